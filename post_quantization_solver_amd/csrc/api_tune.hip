// The C ABI's operators of a tuning step (include/mpq.h): argument checks on
// the host, then launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>
#include <algorithm>
#include <utility>
#include <vector>

#include "../../include/mpq.h"
#include "adamw.h"

using namespace mpq;

namespace {

constexpr size_t ALIGN = 256;
constexpr uint64_t PLAN_MAGIC = 0x4d505141444d5731ull;   // "MPQADMW1"
constexpr int64_t MAX_TENSORS = 1 << 16, MAX_ELEMENTS = (int64_t)1 << 40;

int status_of(hipError_t e) { return e == hipSuccess ? MPQ_OK : hip_status(e); }

bool plain_dtype(int dtype) { return dtype == MPQ_BF16 || dtype == MPQ_FP16 || dtype == MPQ_FP32; }
int64_t element(int dtype) { return dtype == MPQ_FP32 ? 4 : 2; }

struct PlanLayout {
  size_t partial, tensors, first, owner, total;
};
size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
PlanLayout plan_layout(int64_t count, int64_t units) {
  PlanLayout P;
  P.partial = up(CTL_WORDS * sizeof(uint32_t));
  const int64_t launches = std::max<int64_t>(1, (count + ADAMW_LAUNCH - 1) / ADAMW_LAUNCH);
  P.tensors = P.partial + up((size_t)launches * ADAMW_NORM_GROUPS * sizeof(double));
  P.first = P.tensors + up((size_t)count * sizeof(AdamwTensor));
  P.owner = P.first + up((size_t)(count + 1) * sizeof(int64_t));
  P.total = P.owner + up((size_t)units * sizeof(int32_t));
  return P;
}

// Counts and places; units and the moments' elements of tensors that are in order.
bool plan_sizes(const mpq_adamw_tensor* t, int64_t count, int64_t* units, int64_t* elements) {
  *units = *elements = 0;
  if (count < 0 || count > MAX_TENSORS || (count > 0 && !t)) return false;
  for (int64_t k = 0; k < count; ++k) {
    if (t[k].count < 0 || t[k].count > MAX_ELEMENTS || t[k].at < *elements || t[k].at > MAX_ELEMENTS ||
        t[k].at % ADAMW_BLOCK != 0)
      return false;
    *elements = t[k].at + (t[k].count + ADAMW_BLOCK - 1) / ADAMW_BLOCK * ADAMW_BLOCK;
    if (*elements > MAX_ELEMENTS) return false;
    *units += adamw_units(t[k].count);
  }
  return true;
}

AdamwTable table_of(const mpq_adamw_plan_t& plan) {
  const PlanLayout P = plan_layout(plan.count, plan.units);
  char* base = static_cast<char*>(plan.table);
  AdamwTable T;
  T.control = reinterpret_cast<uint32_t*>(base);
  T.partial = reinterpret_cast<double*>(base + P.partial);
  T.tensors = reinterpret_cast<const AdamwTensor*>(base + P.tensors);
  T.first = reinterpret_cast<const int64_t*>(base + P.first);
  T.owner = reinterpret_cast<const int32_t*>(base + P.owner);
  T.count = plan.count;
  T.units = plan.units;
  return T;
}

int make_plan(const mpq_adamw_tensor* t, int64_t count, void* plan, size_t plan_bytes, hipStream_t st,
              mpq_adamw_plan_t* out) {
  int64_t units, elements;
  if (!plan_sizes(t, count, &units, &elements)) return MPQ_ESHAPE;
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  for (int64_t k = 0; k < count; ++k) {
    if (!plain_dtype(t[k].dtype) || !(t[k].lr >= 0.f) || !isfinite(t[k].lr) || !(t[k].weight_decay >= 0.f) ||
        !isfinite(t[k].weight_decay) || t[k].reserved != 0)
      return MPQ_EPARAM;
    if (t[k].count == 0) continue;
    if (!t[k].param) return MPQ_ENULL;
    const uintptr_t p = reinterpret_cast<uintptr_t>(t[k].param);
    if (p % element(t[k].dtype) != 0) return MPQ_EPARAM;
    spans.emplace_back(p, p + (uintptr_t)(t[k].count * element(t[k].dtype)));
  }
  std::sort(spans.begin(), spans.end());
  for (size_t k = 1; k < spans.size(); ++k)
    if (spans[k].first < spans[k - 1].second) return MPQ_EPARAM;
  const PlanLayout P = plan_layout(count, units);
  if (!plan || reinterpret_cast<uintptr_t>(plan) % ALIGN != 0 || plan_bytes < P.total) return MPQ_EWORKSPACE;
  std::vector<char> image(P.total, 0);   // (the counters begin at zero)
  AdamwTensor* tensors = reinterpret_cast<AdamwTensor*>(image.data() + P.tensors);
  int64_t* first = reinterpret_cast<int64_t*>(image.data() + P.first);
  int32_t* owner = reinterpret_cast<int32_t*>(image.data() + P.owner);
  int64_t at = 0;
  for (int64_t k = 0; k < count; ++k) {
    tensors[k] = {t[k].param, t[k].count, t[k].at, t[k].lr, t[k].weight_decay, t[k].dtype, 0};
    first[k] = at;
    const int64_t u = adamw_units(t[k].count);
    std::fill(owner + at, owner + at + u, (int32_t)k);
    at += u;
  }
  first[count] = at;
  hipError_t e = hipMemcpyAsync(plan, image.data(), P.total, hipMemcpyHostToDevice, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_status(e);
  out->count = count;
  out->units = units;
  out->elements = elements;
  out->table = plan;
  out->magic = PLAN_MAGIC;
  return MPQ_OK;
}

int state_ok(const mpq_adamw_state& s, int64_t elements) {
  if (s.bits != 8 && s.bits != 32) return MPQ_EPARAM;
  if (s.elements < elements || s.elements < 0 || s.elements > MAX_ELEMENTS) return MPQ_ESHAPE;
  if (elements > 0 && (!s.m || !s.v || (s.bits == 8 && (!s.m_scale || !s.v_scale)))) return MPQ_ENULL;
  if (reinterpret_cast<uintptr_t>(s.m) % 16 != 0 || reinterpret_cast<uintptr_t>(s.v) % 16 != 0) return MPQ_EWORKSPACE;
  return MPQ_OK;
}

}  // namespace

extern "C" {

size_t mpq_adamw_plan_bytes(const mpq_adamw_tensor* tensors, int64_t count) {
  int64_t units, elements;
  return plan_sizes(tensors, count, &units, &elements) ? plan_layout(count, units).total : 0;
}

int mpq_adamw_plan(const mpq_adamw_tensor* tensors, int64_t count, void* plan, size_t plan_bytes, void* stream,
                   mpq_adamw_plan_t* out) {
  try {
    if (!out || (count > 0 && !tensors)) return MPQ_ENULL;
    return make_plan(tensors, count, plan, plan_bytes, static_cast<hipStream_t>(stream), out);
  } catch (...) {
    return MPQ_EHOST;
  }
}

int mpq_adamw(const mpq_adamw_plan_t* plan, const void* const* grads, const mpq_adamw_options* options,
              const mpq_adamw_state* state, void* stream) {
  if (!plan || !options || !state) return MPQ_ENULL;
  if (plan->magic != PLAN_MAGIC) return MPQ_EPARAM;
  const mpq_adamw_options& o = *options;
  if (!(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) || !(o.eps > 0.0) || !isfinite((float)o.eps) ||
      (float)o.eps == 0.f || !isfinite(o.grad_scale) || !(o.max_norm >= 0.0) ||
      !(o.lr_scale >= 0.0) || !isfinite((float)o.lr_scale))
    return MPQ_EPARAM;
  const int rc = state_ok(*state, plan->elements);
  if (rc) return rc;
  if (!state->step || (plan->units > 0 && !grads)) return MPQ_ENULL;
  AdamwCall A;
  A.table = table_of(*plan);
  A.grads = grads;
  A.small = state->bits == 8;
  A.clip = o.max_norm > 0.0;
  A.grad_scale = o.grad_scale;
  A.max_norm = o.max_norm;
  A.lr_scale = (float)o.lr_scale;
  A.lr_factor = o.lr_factor;
  A.beta1 = o.beta1;
  A.beta2 = o.beta2;
  A.eps = (float)o.eps;
  A.seed = state->seed;
  A.step = state->step;
  A.m = state->m;
  A.v = state->v;
  A.m_scale = state->m_scale;
  A.v_scale = state->v_scale;
  A.norm = o.norm;
  return status_of(launch_adamw(A, static_cast<hipStream_t>(stream)));
}

int mpq_adamw_moments(const mpq_adamw_state* state, float* m, float* v, void* stream) {
  if (!state) return MPQ_ENULL;
  if (state->bits != 8) return MPQ_EPARAM;
  if (state->elements % ADAMW_BLOCK != 0) return MPQ_ESHAPE;
  const int rc = state_ok(*state, state->elements);
  if (rc) return rc;
  if (state->elements > 0 && (!m || !v)) return MPQ_ENULL;
  if (reinterpret_cast<uintptr_t>(m) % 16 != 0 || reinterpret_cast<uintptr_t>(v) % 16 != 0) return MPQ_EWORKSPACE;
  return status_of(launch_adamw_moments(static_cast<const uint8_t*>(state->m), static_cast<const uint8_t*>(state->v),
                                        state->m_scale, state->v_scale, state->elements, m, v,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
