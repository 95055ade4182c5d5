// The C ABI's operators around a solved layer (include/mpq.h): argument checks
// on the host, then launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/mpq.h"
#include "qlayer.h"

using namespace mpq;

namespace {

constexpr size_t ALIGN = 256;

bool dtype_ok(int dtype) { return dtype == MPQ_BF16 || dtype == MPQ_FP16 || dtype == MPQ_FP32; }

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && reinterpret_cast<uintptr_t>(ws) % ALIGN == 0 && have >= need);
}

// Sizes of valid shapes are never 0, which means shapes out of range.
size_t sized(size_t bytes) { return bytes > ALIGN ? bytes : ALIGN; }

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

constexpr int64_t Q_MAX_M = (int64_t)1 << 24, Q_MAX_N = 65536, Q_MAX_T = (int64_t)1 << 22;

// A layer's shapes and format (no pointers).
int layer_shape(QLayer& L, int64_t m, int64_t n, int64_t K, int64_t d, int64_t group, int kind) {
  if (d != 1 && d != 8) return MPQ_EUNSUPPORTED;
  if (m < 0 || m > Q_MAX_M || n < 1 || n > Q_MAX_N || n % d != 0) return MPQ_ESHAPE;
  if (d == 1 ? K < 2 || K > 64 : K < 1 || K > 65536) return MPQ_ESHAPE;
  if (group < 0) return MPQ_EPARAM;
  if (group > 0 && d != 1) return MPQ_EUNSUPPORTED;
  L = QLayer{};
  L.fmt = d == 1 ? (K <= 16 ? QF_NIB : QF_BYTE) : kind == MPQ_CB_E8_PREFIX ? QF_E8 : QF_VEC;
  L.m = m;
  L.n = n;
  L.K = (int)K;
  L.tiles = (int)((m + 15) / 16);
  L.chunks = (int)((n + q_chunk(L.fmt) - 1) / q_chunk(L.fmt));
  // (a thread per 16 bytes lays them out, and a grid has fewer than 2^32)
  if ((int64_t)L.tiles * L.chunks >= (int64_t)1 << 26) return MPQ_ESHAPE;
  L.group = group > 0 && group < n ? group : n;
  L.G = (int)((n + L.group - 1) / L.group);
  return MPQ_OK;
}

int layer_of(QLayer& L, const void* packed, int64_t m, int64_t n, const mpq_codebook* cb, const float* scale,
             const float* offset, int64_t group) {
  CbTables T;
  int rc = prepared_tables(cb, T);
  if (rc) return rc;
  if ((rc = layer_shape(L, m, n, cb->K, cb->d, group, cb->kind))) return rc;
  if (!(cb->magic & CB_NARROW)) return MPQ_EUNSUPPORTED;
  L.packed = static_cast<const uint4*>(packed);
  L.scale = scale;
  L.offset = offset;
  L.levels = T.levels;
  L.uniform = (cb->magic & CB_EVEN) != 0;
  L.lut = T.pk_lut;
  L.map = T.pk_map;
  L.e32 = T.e32;
  if (L.fmt == QF_E8) {
    L.pairs = q_e8_pairs(cb->K);
    L.lut_entries = (int)cb->K - L.pairs;
  }
  return MPQ_OK;
}

// What the gradients' grids of 256 threads a workgroup take (fewer than 2^32 in
// all): tiles of 64 x 64 of du and x; 16 entries of the affine a workgroup beside
// d bias, where the contraction takes the layer in one piece.
bool grad_fits(const QLayer& L, int64_t t) {
  const int64_t most = (int64_t)1 << 24;
  return ((L.m + 63) / 64 + (L.n + 63) / 64) * ((t + 63) / 64) < most &&
         (L.group % Q_CONTRACT != 0 || (L.m * L.G + 15) / 16 + (L.m + 255) / 256 < most);
}

// Enough for every combination of outputs and activation.
size_t grad_workspace(QLinearGrad A) {
  A.act = ACT_RELU;
  A.need_dx = A.need_dlayer = true;
  return q_grad_workspace(A);
}

}  // namespace

namespace mpq {
int q_layer_shape(QLayer& L, int64_t m, int64_t n, int64_t K, int64_t d, int64_t group, int kind) {
  return layer_shape(L, m, n, K, d, group, kind);
}
int q_layer_of(QLayer& L, const void* packed, int64_t m, int64_t n, const mpq_codebook* cb, const float* scale,
               const float* offset, int64_t group) {
  return layer_of(L, packed, m, n, cb, scale, offset, group);
}
}  // namespace mpq

extern "C" {

size_t mpq_pack_bytes(int64_t m, int64_t n, int64_t K, int64_t d) {
  QLayer L;
  return layer_shape(L, m, n, K, d, 0, MPQ_CB_GENERIC) == MPQ_OK ? sized(q_packed_bytes(L)) : 0;
}

int mpq_pack(const int32_t* codes, int64_t m, int64_t n, const mpq_codebook* cb, void* packed, size_t packed_bytes,
             void* stream) {
  QLayer L;
  const int rc = layer_of(L, packed, m, n, cb, nullptr, nullptr, 0);
  if (rc) return rc;
  if (m == 0) return MPQ_OK;
  if (!codes) return MPQ_ENULL;
  if (!workspace_ok(packed, packed_bytes, q_packed_bytes(L))) return MPQ_EWORKSPACE;
  return status_of(launch_q_pack(codes, L, packed, static_cast<hipStream_t>(stream)));
}

size_t mpq_linear_workspace_bytes(int dtype, int64_t t, int64_t m, int64_t n, int64_t K, int64_t d, int64_t group) {
  QLinearArgs A = {};
  if (!dtype_ok(dtype) || t < 0 || t >= Q_MAX_T || layer_shape(A.L, m, n, K, d, group, MPQ_CB_GENERIC) != MPQ_OK)
    return 0;
  A.dtype = dtype;
  A.t = t;
  return sized(q_linear_workspace(A));
}

int mpq_linear(const void* x, int dtype, int64_t t, int64_t ldx, const void* packed, int64_t m, int64_t n,
               const mpq_codebook* cb, const float* scale, const float* offset, int64_t group, const float* bias,
               int act, const void* residual, int64_t ldr, void* y, int64_t ldy, void* pre, int64_t ldp,
               void* workspace, size_t ws_bytes, void* stream) {
  QLinearArgs A = {};
  const int rc = layer_of(A.L, packed, m, n, cb, scale, offset, group);
  if (rc) return rc;
  if (!dtype_ok(dtype) || act < MPQ_ACT_NONE || act > MPQ_ACT_SILU) return MPQ_EPARAM;
  if (t < 0 || t >= Q_MAX_T || ldx < n || ldy < m || (residual && ldr < m) || (pre && ldp < m)) return MPQ_ESHAPE;
  if (t == 0 || m == 0) return MPQ_OK;
  if (!x || !packed || !scale || !y) return MPQ_ENULL;
  A.x = x;
  A.ldx = ldx;
  A.dtype = dtype;
  A.t = t;
  A.bias = bias;
  A.act = act;
  A.res = residual;
  A.ldres = ldr;
  A.y = y;
  A.ldy = ldy;
  A.pre = pre;
  A.ldpre = ldp;
  if (!workspace_ok(packed, SIZE_MAX, 1)) return MPQ_EWORKSPACE;
  if (!workspace_ok(workspace, ws_bytes, q_linear_workspace(A))) return MPQ_EWORKSPACE;
  return status_of(launch_q_linear(A, workspace, static_cast<hipStream_t>(stream)));
}

size_t mpq_linear_backward_workspace_bytes(int dtype, int64_t t, int64_t m, int64_t n, int64_t K, int64_t d,
                                           int64_t group) {
  QLinearGrad A = {};
  if (!dtype_ok(dtype) || t < 0 || t >= Q_MAX_T || layer_shape(A.L, m, n, K, d, group, MPQ_CB_GENERIC) != MPQ_OK ||
      !grad_fits(A.L, t))
    return 0;
  A.dtype = dtype;
  A.t = t;
  return sized(grad_workspace(A));
}

int mpq_linear_backward(const void* dy, int64_t lddy, const void* x, int dtype, int64_t t, int64_t ldx,
                        const void* packed, int64_t m, int64_t n, const mpq_codebook* cb, const float* scale,
                        const float* offset, int64_t group, int act, const void* pre, int64_t ldp, void* dx,
                        int64_t lddx, float* dscale, float* doffset, float* dbias, void* workspace, size_t ws_bytes,
                        void* stream) {
  QLinearGrad A = {};
  const int rc = layer_of(A.L, packed, m, n, cb, scale, offset, group);
  if (rc) return rc;
  const bool need_dlayer = dscale || doffset || dbias;
  if (!dtype_ok(dtype) || act < MPQ_ACT_NONE || act > MPQ_ACT_SILU) return MPQ_EPARAM;
  if (t < 0 || t >= Q_MAX_T || lddy < m || ldx < n || (act != MPQ_ACT_NONE && ldp < m) || (dx && lddx < n) ||
      !grad_fits(A.L, t))
    return MPQ_ESHAPE;
  if (need_dlayer && m > 0 && (!dscale || !doffset || !dbias)) return MPQ_ENULL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (m == 0 || t == 0) {
    // nothing to sum: gradients of zero
    hipError_t e = hipSuccess;
    if (t == 0 && m > 0 && need_dlayer) {
      e = launch_fill_i32(reinterpret_cast<int32_t*>(dscale), m * A.L.G, 0, st);
      if (e == hipSuccess) e = launch_fill_i32(reinterpret_cast<int32_t*>(doffset), m * A.L.G, 0, st);
      if (e == hipSuccess) e = launch_fill_i32(reinterpret_cast<int32_t*>(dbias), m, 0, st);
    }
    if (e == hipSuccess && t > 0 && dx) e = launch_q_zero_rows(dx, t, n, lddx, dtype, st);   // a layer without rows
    return status_of(e);
  }
  if (!dy || !x || !packed || !scale || (act != MPQ_ACT_NONE && !pre)) return MPQ_ENULL;
  A.dy = dy;
  A.lddy = lddy;
  A.x = x;
  A.ldx = ldx;
  A.pre = pre;
  A.ldpre = ldp;
  A.dtype = dtype;
  A.act = act;
  A.t = t;
  A.need_dx = dx != nullptr;
  A.need_dlayer = need_dlayer;
  A.dx = dx;
  A.lddx = lddx;
  A.dscale = dscale;
  A.doffset = doffset;
  A.dbias = dbias;
  if (!workspace_ok(packed, SIZE_MAX, 1)) return MPQ_EWORKSPACE;
  if (!workspace_ok(workspace, ws_bytes, grad_workspace(A))) return MPQ_EWORKSPACE;
  return status_of(launch_q_grad(A, workspace, st));
}

size_t mpq_token_logprobs_workspace_bytes(int dtype, int64_t t, int64_t V, int top) {
  LogitArgs A;
  if (logit_args(A, nullptr, dtype, t, V, V, top, 0) != MPQ_OK) return 0;
  return sized(logit_workspace(A));
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
  return sized(logit_workspace(A));
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
