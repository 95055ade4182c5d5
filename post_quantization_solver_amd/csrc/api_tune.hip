// The C ABI's operators of a tuning step (include/mpq.h): argument checks on
// the host, then launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <string.h>
#include <algorithm>
#include <utility>
#include <vector>

#include "../../include/mpq.h"
#include "adamw.h"
#include "head.h"

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

constexpr int64_t HEAD_MAX_T = (int64_t)1 << 22, HEAD_MAX_M = (int64_t)1 << 24, HEAD_MAX_N = 65536;

// A matrix's shapes.
int matrix_shape(QLayer& L, int64_t m, int64_t n) {
  if (m < 0 || m > HEAD_MAX_M || n < 1 || n > HEAD_MAX_N) return MPQ_ESHAPE;
  L = QLayer{};
  L.fmt = QF_VEC;
  L.m = m;
  L.n = n;
  L.tiles = (int)((m + 15) / 16);
  L.group = n;
  L.G = 1;
  return MPQ_OK;
}

// Grids of fewer than 2^32 threads: a workgroup per token, tiles of dx of 64 x 64 at least.
bool head_fits(const HeadArgs& A) {
  return A.t >= 0 && A.t < HEAD_MAX_T && A.L.m >= 1 && (A.t + 63) / 64 * ((A.L.n + 63) / 64) < (int64_t)1 << 24;
}

// Enough for every combination of outputs.
size_t head_bytes(HeadArgs A) {
  A.need_dx = A.need_dhead = true;
  A.t = std::max<int64_t>(A.t, 1);
  const size_t b = head_workspace(A);
  return b > ALIGN ? b : ALIGN;
}

// The arguments that both kinds of head have.
int head_call(HeadArgs& A, int dtype, const void* x, int64_t t, int64_t ldx, const float* bias, const int32_t* targets,
              const float* weights, float* loss, void* dx, int64_t lddx, void* workspace, size_t ws_bytes, hipStream_t st,
              float* dscale, float* doffset, float* dbias, void* dW, int64_t lddw) {
  if (!plain_dtype(dtype)) return MPQ_EPARAM;
  A.t = t;
  if (!head_fits(A) || ldx < A.L.n || (dx && lddx < A.L.n) || (dW && lddw < A.L.n)) return MPQ_ESHAPE;
  if (A.need_dhead && (!dbias || (A.dense ? !dW : !dscale || !doffset))) return MPQ_ENULL;
  if (t == 0) {   // nothing to sum
    hipError_t e = hipSuccess;
    if (A.need_dhead) {
      if (dscale) e = launch_fill_i32(reinterpret_cast<int32_t*>(dscale), A.L.m * A.L.G, 0, st);
      if (e == hipSuccess && doffset) e = launch_fill_i32(reinterpret_cast<int32_t*>(doffset), A.L.m * A.L.G, 0, st);
      if (e == hipSuccess) e = launch_fill_i32(reinterpret_cast<int32_t*>(dbias), A.L.m, 0, st);
      if (e == hipSuccess && dW) e = launch_q_zero_rows(dW, A.L.m, A.L.n, lddw, dtype, st);
    }
    return status_of(e);
  }
  if (!x || !targets || !loss) return MPQ_ENULL;
  A.dtype = dtype;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % ALIGN != 0 || ws_bytes < head_bytes(A)) return MPQ_EWORKSPACE;
  A.x = x;
  A.ldx = ldx;
  A.bias = bias;
  A.targets = targets;
  A.weights = weights;
  A.loss = loss;
  A.need_dx = dx != nullptr;
  A.dx = dx;
  A.lddx = lddx;
  A.dscale = dscale;
  A.doffset = doffset;
  A.dbias = dbias;
  A.dW = dW;
  A.lddw = lddw;
  return status_of(launch_head(A, workspace, st));
}

}  // namespace

extern "C" {

size_t mpq_linear_cross_entropy_workspace_bytes(int dtype, int64_t t, int64_t m, int64_t n, int64_t K, int64_t d,
                                                int64_t group) {
  HeadArgs A = {};
  if (!plain_dtype(dtype) || q_layer_shape(A.L, m, n, K, d, group, MPQ_CB_GENERIC) != MPQ_OK) return 0;
  A.dtype = dtype;
  A.t = t;
  return head_fits(A) ? head_bytes(A) : 0;
}

int mpq_linear_cross_entropy(const void* x, int dtype, int64_t t, int64_t ldx, const void* packed, int64_t m, int64_t n,
                             const mpq_codebook* cb, const float* scale, const float* offset, int64_t group,
                             const float* bias, const int32_t* targets, const float* weights, float* loss, void* dx,
                             int64_t lddx, float* dscale, float* doffset, float* dbias, void* workspace, size_t ws_bytes,
                             void* stream) {
  HeadArgs A = {};
  const int rc = q_layer_of(A.L, packed, m, n, cb, scale, offset, group);
  if (rc) return rc;
  if (t != 0 && (!packed || !scale)) return MPQ_ENULL;
  if (reinterpret_cast<uintptr_t>(packed) % ALIGN != 0) return MPQ_EWORKSPACE;
  A.need_dhead = dscale || doffset || dbias;
  return head_call(A, dtype, x, t, ldx, bias, targets, weights, loss, dx, lddx, workspace, ws_bytes,
                   static_cast<hipStream_t>(stream), dscale, doffset, dbias, nullptr, n);
}

size_t mpq_matrix_cross_entropy_workspace_bytes(int dtype, int64_t t, int64_t m, int64_t n) {
  HeadArgs A = {};
  if (!plain_dtype(dtype) || matrix_shape(A.L, m, n) != MPQ_OK) return 0;
  A.dense = true;
  A.dtype = dtype;
  A.t = t;
  return head_fits(A) ? head_bytes(A) : 0;
}

int mpq_matrix_cross_entropy(const void* x, int dtype, int64_t t, int64_t ldx, const void* W, int64_t ldw, int64_t m,
                             int64_t n, const float* bias, const int32_t* targets, const float* weights, float* loss,
                             void* dx, int64_t lddx, void* dW, int64_t lddw, float* dbias, void* workspace,
                             size_t ws_bytes, void* stream) {
  HeadArgs A = {};
  const int rc = matrix_shape(A.L, m, n);
  if (rc) return rc;
  if (ldw < n) return MPQ_ESHAPE;
  if (t != 0 && !W) return MPQ_ENULL;
  A.dense = true;
  A.W = W;
  A.ldw = ldw;
  A.need_dhead = dW || dbias;
  return head_call(A, dtype, x, t, ldx, bias, targets, weights, loss, dx, lddx, workspace, ws_bytes,
                   static_cast<hipStream_t>(stream), nullptr, nullptr, dbias, dW, lddw);
}

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
  // (the reciprocal of an eps below float32's normal range is infinite: times a first moment of 0, NaN)
  if (!(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) || !((float)o.eps >= FLT_MIN) ||
      !isfinite((float)o.eps) || !isfinite(o.grad_scale) || !(o.max_norm >= 0.0) || !(o.lr_scale >= 0.0) ||
      !isfinite((float)o.lr_scale))
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
