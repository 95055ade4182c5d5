// The C ABI's operators around a solved layer (include/mpq.h): argument checks
// on the host, then launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/mpq.h"
#include "internal.h"

using namespace mpq;

namespace {

constexpr size_t ALIGN = 256;

bool dtype_ok(int dtype) { return dtype == MPQ_BF16 || dtype == MPQ_FP16 || dtype == MPQ_FP32; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && reinterpret_cast<uintptr_t>(ws) % ALIGN == 0 && have >= need);
}

int status_of(hipError_t e) { return e == hipSuccess ? MPQ_OK : hip_status(e); }

// Rows of logits with `top` alternatives or a teacher's list of k.
int logit_args(LogitArgs& A, const void* z, int dtype, int64_t t, int64_t V, int64_t ldz, int top, int k) {
  if (!dtype_ok(dtype)) return MPQ_EPARAM;
  if (t < 0 || V < 1 || V > LOGIT_MAX_V || ldz < V || top < 0 || top > LOGIT_MAX_TOP || k < 0 || k > LOGIT_MAX_TOP)
    return MPQ_ESHAPE;
  A = LogitArgs{};
  A.z = z;
  A.ldz = ldz;
  A.dtype = dtype;
  A.t = t;
  A.V = V;
  A.top = top;
  A.k = k;
  logit_split(A);
  if (t > (INT32_MAX / (int64_t)A.S)) return MPQ_ESHAPE;
  return MPQ_OK;
}

}  // namespace

extern "C" {

size_t mpq_token_logprobs_workspace_bytes(int dtype, int64_t t, int64_t V, int top) {
  LogitArgs A;
  if (logit_args(A, nullptr, dtype, t, V, V, top, 0) != MPQ_OK) return 0;
  return logit_workspace(A);
}

int mpq_token_logprobs(const void* logits, int dtype, int64_t t, int64_t V, int64_t ld, const int32_t* tokens, int top,
                       float* logprob, float* entropy, float* lse, int32_t* top_ids, float* top_logprobs,
                       void* workspace, size_t ws_bytes, void* stream) {
  LogitArgs A;
  const int rc = logit_args(A, logits, dtype, t, V, ld, top, 0);
  if (rc) return rc;
  if (t == 0) return MPQ_OK;
  if (!logits || (logprob && !tokens)) return MPQ_ENULL;
  if (!workspace_ok(workspace, ws_bytes, logit_workspace(A))) return MPQ_EWORKSPACE;
  A.c = (float)1.4426950408889634074;
  return status_of(launch_token_logprobs(A, tokens, logprob, entropy, lse, top_ids, top_logprobs, workspace,
                                         static_cast<hipStream_t>(stream)));
}

size_t mpq_distill_workspace_bytes(int dtype, int64_t t, int64_t V, int k) {
  LogitArgs A;
  if (logit_args(A, nullptr, dtype, t, V, V, 0, k) != MPQ_OK) return 0;
  return logit_workspace(A);
}

int mpq_distill(const void* logits, int dtype, int64_t t, int64_t V, int64_t ld, const int32_t* ids,
                const float* teacher, int k, float temperature, int tail, const float* weights, float* loss,
                void* grad, int64_t ldg, void* workspace, size_t ws_bytes, void* stream) {
  LogitArgs A;
  const int rc = logit_args(A, logits, dtype, t, V, ld, 0, k);
  if (rc) return rc;
  if (grad && ldg < V) return MPQ_ESHAPE;
  if (!(temperature > 0.f) || !isfinite(temperature) || (tail && temperature != 1.f)) return MPQ_EPARAM;
  if (t == 0) return MPQ_OK;
  if (!logits || !loss || (k > 0 && (!ids || !teacher))) return MPQ_ENULL;
  if (!workspace_ok(workspace, ws_bytes, logit_workspace(A))) return MPQ_EWORKSPACE;
  const double invT = 1.0 / (double)temperature;
  A.c = (float)(1.4426950408889634074 * invT);
  if (!isfinite(A.c) || !(A.c > 0.f)) return MPQ_EPARAM;
  A.ids = ids;
  A.weights = weights;
  return status_of(launch_distill(A, teacher, invT, tail != 0, loss, grad, ldg, workspace,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"
