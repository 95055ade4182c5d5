// Softmax cross entropy of an output head in pieces of the vocabulary, and its
// gradients; logits are kept only where they take up to 128 MB.
//
// Mathematics.  z_tv = a_v s_tv + o_v X_t + b_v with s = x e^T over the head's
// entries and X_t = sum_j x_tj (a matrix or column groups: s = x W^T alone); r the
// target, w the token's weight:
//   R_t = log sum_{v != r} exp z_tv,     loss = w log(1 + exp(R_t - z_tr)),
//   dz_tv = w exp(z_tv - lse_t), v != r,  dz_tr = -w / (1 + exp(z_tr - R_t)),
//   dx = dz W,  db_v = sum_t dz_tv,  da_v = sum_t dz_tv s_tv,  do_v = sum_t dz_tv X_t;
//   a matrix: dW = dz^T x; column groups: dW's sums with the entries and without.
// With the target's term apart a small loss, and the gradient of a token that is
// all but certain, keep their relative accuracy.  With one affine per row the
// layer's gradients are sums over what the logits are made of: no product of
// their own.
//
// Order.  The vocabulary goes in pieces of some thousand rows: the piece's
// operand planes, its logits, and of each token the largest and the sum of the
// exponentials.  Once all pieces have gone by (R is known) they come again for the
// gradients: logits once more, dz, its products.  Logits that fit are kept instead, and
// multiplied once; for the gradient of a matrix or of column groups, where dz^T's rows have a
// factor each that takes all tokens to know, a piece's are formed again in memory.
//
// Bound.  Many tokens: the products, see headgemm.hip (2048 x 128256 x 4096 E8: 1.64 ms for
// the loss, 5.34 with the gradients of the layer's affine and of x, of which 0.22 and 0.46 lay
// the planes out at 5.4 TB/s).  Logits that are kept (509 x 50257 x 2048, groups of 128: 0.91
// to 0.94 ms): the products take 0.67, planes 0.11, dz 0.07, its bounds 0.02.  A token (32000 x
// 4096 E8: 37 us): the few-row product of the codes, 26.
#include <string.h>
#include <math.h>
#include <algorithm>
#include "head.h"

namespace mpq {

namespace {

constexpr size_t HALIGN = 256;
inline size_t up(size_t x) { return (x + HALIGN - 1) / HALIGN * HALIGN; }
inline int64_t up64(int64_t x) { return (x + 63) / 64 * 64; }
inline int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
struct Carve {
  char* base;
  size_t at = 0;
  template <typename P>
  P* take(size_t bytes) {
    P* p = base ? reinterpret_cast<P*>(base + at) : nullptr;
    at += up(bytes);
    return p;
  }
};

// Tokens whose input gradient comes straight from the packed codes.  Measured, whole calls with
// gradients, 4 tokens so | 5 through planes: E8 128256 x 4096 323 | 600 us, 32000 x 2048 72 | 97;
// 4 bits 32000 x 4096 102 | 165, groups of 128 117 | 232; 6 bits 32000 x 2048 80 | 114.  (One
// token: 186, 54, 65, 72, 62.)  Eight would read and decode the codes twice.
constexpr int64_t H_FEW = 4;
// What logits that are kept should take (half of the last-level cache); a piece's planes, and
// its dz; the planes of a head whose logits are kept, which both passes read; rows that a piece
// has at least.  Measured: pieces of 64, 128, 256, 512 MB (2048 x 128256 x 4096 E8 with
// gradients) 5.84, 5.55, 5.35, 5.27 ms, the last for twice the workspace.  Kept logits' planes
// in pieces of 256 | 512 | 1024 MB, where those are more than one they are laid out twice: 412 MB
// (509 x 50257 x 2048, groups of 128) 1100 | 934 | 934 us, 512 MB (300 x 32001 x 8000 bfloat16,
// not in place) 626 | 508 | 508, 524 MB (333 x 64000 x 2048 float32) 1840 | 1535 | 1535, 823 MB
// (512 x 50257 x 8192 E8) 1474 | 1340 | 1017, 1.6 GB (256 x 100000 x 4096, groups of 128)
// 2970 | 2700 | 2580: 512 MB take in all of the heads that vocabularies of some 50000 and kept
// logits mostly go with, and twice that is workspace which every such call would hold.
constexpr int64_t H_BYTES = (int64_t)128 << 20, H_PIECE = (int64_t)256 << 20, H_PLANES = (int64_t)512 << 20, H_ROWS = 1024;

// ------------------------------------------------------------------ tokens

struct TokenArgs {
  const void* x; int64_t ldx;
  int dtype;
  int64_t t, n, V;
  const int32_t* targets;
  const float* weights;
  bool vec;                           // rows of x four elements at a time
  float *weight, *sum, *target_z;     // the weight (0: the row is not read), X, the target's logit
  uint32_t* rowmax;
  uint16_t* planes; int64_t plane;    // float16 terms, operand order of Kp columns
  int terms; int64_t Kp;
  bool raw;                           // bfloat16 as it is, in place of terms
  bool frags;                         // in the few-row product's order
  uint16_t* again; int64_t plane_again, Kp_again;   // terms in operand order beside them (nullptr: none)
  float* ones;                        // V ones, or nullptr
  const float* scale; float* fpart;   // the largest of V scales, in 64 parts (nullptr: not wanted)
};

__device__ __forceinline__ float token_weight(const TokenArgs& A, int64_t t) {
  return t < A.t && A.targets[t] >= 0 ? (A.weights ? A.weights[t] : 1.f) : 0.f;
}

// The larger magnitude, by its bits (NaN over everything).
__device__ __forceinline__ float bits_max(float a, float b) { return __uint_as_float(max(abs_bits(a), abs_bits(b))); }

// A workgroup per row of the planes: the tokens' rows, zeros for those that are
// not read and behind the last.
__global__ __launch_bounds__(256) void head_token_kernel(TokenArgs A) {
  __shared__ float red[2][4];
  const int64_t row = blockIdx.x, rows = (A.t + 15) / 16 * 16;
  const int lane = threadIdx.x & 63, wave = wave_id();
  if (row >= rows) {   // the workgroups behind them
    const int64_t k = row - rows;
    if (A.fpart && k < 64) {
      float top = 0.f;
      for (int64_t i = k * 256 + threadIdx.x; i < A.V; i += 64 * 256) top = bits_max(top, A.scale[i]);
      for (int o = 32; o; o >>= 1) top = bits_max(top, shfl_xor_f(top, o));
      if (lane == 0) red[0][wave] = top;
      __syncthreads();
      if (threadIdx.x == 0) A.fpart[k] = bits_max(bits_max(red[0][0], red[0][1]), bits_max(red[0][2], red[0][3]));
      return;
    }
    const int64_t i = (k - (A.fpart ? 64 : 0)) * 256 + threadIdx.x;
    if (i < A.V) A.ones[i] = 1.f;
    return;
  }
  const float w = token_weight(A, row);
  const bool live = w != 0.f;   // (a NaN weight is one)
  auto load8 = [&](int64_t j, float* v) {
    const int have = live ? (int)max((int64_t)0, min((int64_t)8, A.n - j)) : 0;
    load4(A.x, row * A.ldx + j, A.dtype, A.vec, min(have, 4), v);
    load4(A.x, row * A.ldx + j + 4, A.dtype, A.vec, max(have - 4, 0), v + 4);
  };
  uint32_t top = 0;
  float s = 0.f;
  for (int64_t j = threadIdx.x * 8; j < A.n; j += 256 * 8) {
    float v[8];
    load8(j, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s += v[k];
      top = max(top, abs_bits(v[k]));
    }
  }
  for (int o = 32; o; o >>= 1) {
    s += shfl_xor_f(s, o);
    top = max(top, (uint32_t)shfl_xor_i((int)top, o));
  }
  if (lane == 0) {
    red[0][wave] = s;
    red[1][wave] = __uint_as_float(top);
  }
  __syncthreads();
  top = 0;
  for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(red[1][k]));
  if (threadIdx.x == 0 && row < A.t) {
    A.weight[row] = w;
    A.sum[row] = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    A.rowmax[row] = top;
    A.target_z[row] = __uint_as_float(0x7fc00000u);   // a target past the vocabulary stays NaN
  }
  const float f = pow2(pow2_shift(top));
  for (int64_t j = threadIdx.x * 8; j < A.Kp; j += 256 * 8) {
    float v[8];
    load8(j, v);
    v4u o[2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[2], b[2];
      f16_terms(v[2 * q] * f, a);
      f16_terms(v[2 * q + 1] * f, b);
      o[0][q] = pack2(a[0], b[0]);
      o[1][q] = pack2(a[1], b[1]);
    }
    if (A.again && j < A.Kp_again) {
      uint16_t* dst = A.again + q_at(row, j, A.Kp_again);
      *reinterpret_cast<v4u*>(dst) = o[0];
      if (A.terms > 1) *reinterpret_cast<v4u*>(dst + A.plane_again) = o[1];
    }
    if (A.raw)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[0][q] = OpBf16::pack(v[2 * q], v[2 * q + 1]);
    uint16_t* dst = A.planes + (A.frags ? ((row >> 4) * (A.Kp >> 5) + (j >> 5)) * 512 + ((j >> 3 & 3) * 16 + (row & 15)) * 8
                                        : q_at(row, j, A.Kp));
    *reinterpret_cast<v4u*>(dst) = o[0];
    if (A.terms > 1) *reinterpret_cast<v4u*>(dst + A.plane) = o[1];
  }
}

// ------------------------------------------------------------------ a matrix's planes

struct DenseArgs {
  const void* W; int64_t ldw;
  int dtype;
  bool vec;
  int64_t m, n, Kp;
  int terms;
  uint32_t* refs;                 // rows' largest magnitudes
  uint16_t* out; int64_t plane;   // m rows of Kp
};

// Rows' largest magnitudes and planes: a wave per row of the planes, which keeps a row of
// up to 2048 columns in registers (longer ones are read again).  32000 x 1024 float32, two
// terms: 66 us for 262 MB, 4 TB/s (a workgroup per row, which reads each twice: 75).
__global__ __launch_bounds__(256) void head_dense_kernel(DenseArgs A) {
  constexpr int HOLD = 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave_id();
  if (row >= (A.m + 15) / 16 * 16) return;
  const bool live = row < A.m;
  auto load8 = [&](int64_t j, float* v) {
    const int have = live ? (int)max((int64_t)0, min((int64_t)8, A.n - j)) : 0;
    if (have == 8 && A.vec) {
      load4(A.W, row * A.ldw + j, A.dtype, true, 4, v);
      load4(A.W, row * A.ldw + j + 4, A.dtype, true, 4, v + 4);
    } else {
      load4(A.W, row * A.ldw + j, A.dtype, false, min(have, 4), v);
      load4(A.W, row * A.ldw + j + 4, A.dtype, false, max(have - 4, 0), v + 4);
    }
  };
  float held[HOLD][8];
  uint32_t top = 0;
#pragma unroll
  for (int h = 0; h < HOLD; ++h) {
    load8((h * 64 + lane) * 8, held[h]);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, abs_bits(held[h][k]));
  }
  for (int64_t j = (HOLD * 64 + lane) * 8; j < A.n; j += 64 * 8) {
    float v[8];
    load8(j, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, abs_bits(v[k]));
  }
  for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)shfl_xor_i((int)top, o));
  if (lane == 0 && live) A.refs[row] = top;
  const float f = pow2(pow2_shift(top));
  auto put = [&](int64_t j, float* v) {
    if (j >= A.Kp) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    put_terms(A.out + q_at(row, j, A.Kp), A.plane, A.terms, v);
    put_terms(A.out + q_at(row, j + 4, A.Kp), A.plane, A.terms, v + 4);
  };
#pragma unroll
  for (int h = 0; h < HOLD; ++h) put((h * 64 + lane) * 8, held[h]);
  for (int64_t j = (HOLD * 64 + lane) * 8; j < A.Kp; j += 64 * 8) {
    float v[8];
    load8(j, v);
    put(j, v);
  }
}

// ------------------------------------------------------------------ a piece's logits

struct Col4 {
  float a[4], o[4], b[4];
};
// (the vectors may begin at any float)
typedef float v4fu __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ Col4 col4(const PieceArgs& A, int64_t i) {
  Col4 C;
  const float mid = A.mid >= 0 ? A.levels[A.mid] : 0.f;
  if (i + 4 <= A.m) {
    v4fu a = {1.f, 1.f, 1.f, 1.f}, o = {0.f, 0.f, 0.f, 0.f}, b = o;
    if (A.a) a = *reinterpret_cast<const v4fu*>(A.a + i);
    if (A.o) o = *reinterpret_cast<const v4fu*>(A.o + i);
    if (A.b) b = *reinterpret_cast<const v4fu*>(A.b + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      C.a[k] = a[k];
      C.o[k] = A.a ? fmaf(a[k], mid, o[k]) : 0.f;
      C.b[k] = b[k];
    }
    return C;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    C.a[k] = 1.f;
    C.o[k] = C.b[k] = 0.f;
    if (i + k >= A.m) continue;
    if (A.a) {
      C.a[k] = A.a[i + k];
      C.o[k] = fmaf(C.a[k], mid, A.o ? A.o[i + k] : 0.f);
    }
    if (A.b) C.b[k] = A.b[i + k];
  }
  return C;
}

// A token's segment of 1024 NQ rows: its largest logit and the sum of the exponentials,
// without the target.
template <int NQ>
__global__ __launch_bounds__(256) void head_stats_kernel(PieceArgs A) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x, i0 = (int64_t)blockIdx.y * (NQ * 1024);
  const int wave = wave_id();
  const int64_t target = (int64_t)A.targets[t] - A.row0;
  const float X = A.sum[t];
  float z[NQ * 4], top = -INFINITY;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int64_t i = i0 + q * 1024 + threadIdx.x * 4;
    const Col4 C = col4(A, i);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < A.m) s = *reinterpret_cast<const float4*>(A.S + t * A.lds + i);
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y = i + k < A.m ? fmaf(C.a[k], v[k], fmaf(C.o[k], X, C.b[k])) : -INFINITY;
      if (i + k == target && i + k < A.m) {
        A.target_z[t] = y;
        y = -INFINITY;
      }
      z[q * 4 + k] = y;
      top = fmaxf(top, y);
    }
  }
  for (int o = 32; o; o >>= 1) top = fmaxf(top, shfl_xor_f(top, o));
  if ((threadIdx.x & 63) == 0) red[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float from = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < NQ * 4; ++k) sum += __builtin_amdgcn_exp2f((z[k] - from) * H_LOG2E);
  for (int o = 32; o; o >>= 1) sum += shfl_xor_f(sum, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) A.part[(int64_t)blockIdx.y * A.t + t] = make_float2(top, (red[0] + red[1]) + (red[2] + red[3]));
}

// A token's loss, and what its gradients take, from the largest of the others' logits, the
// sum of their exponentials about it, and the target's.
struct TokenOut {
  const float* weight;
  float *loss, *row_top, *row_scale, *row_target;
};
__device__ __forceinline__ void finish_token(const TokenOut& A, int64_t t, float top, double s, float zt) {
  const float w = A.weight[t];
  if (w == 0.f) {   // not read
    A.loss[t] = A.row_top[t] = A.row_scale[t] = A.row_target[t] = 0.f;
    return;
  }
  if (!(s == s) || !(zt == zt)) {
    A.row_top[t] = 0.f;
    A.loss[t] = A.row_scale[t] = A.row_target[t] = __uint_as_float(0x7fc00000u);
    return;
  }
  // R - z of the target: log of the others' mass over its own
  const double d = (double)top + log(s) - (double)zt;
  const bool none = zt == -INFINITY;   // (all of them: nothing to move)
  const double rest = none ? 1.0 : d > 0.0 ? 1.0 / (1.0 + exp(-d)) : exp(d) / (1.0 + exp(d));
  const double l = none ? INFINITY : d > 0.0 ? d + log1p(exp(-d)) : log1p(exp(d));
  const float all = fmaxf(top, zt);
  const double total = s * exp((double)top - (double)all) + exp((double)zt - (double)all);
  A.loss[t] = (float)((double)w * l);
  A.row_top[t] = all;
  A.row_scale[t] = all == -INFINITY ? 0.f : (float)((double)w / total);
  A.row_target[t] = all == -INFINITY ? 0.f : (float)(-(double)w * rest);
}

// The segments joined: sixteen tokens a workgroup, sixteen threads each.
__global__ __launch_bounds__(256) void head_join_kernel(const float2* __restrict__ part, int64_t segs, int64_t T,
                                                        const float* __restrict__ target_z, TokenOut O) {
  __shared__ float tops[16][16];
  __shared__ double sums[16][16];
  const int own = threadIdx.x & 15, lane = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * 16 + own, at = min(t, T - 1);
  float top = -INFINITY;
#pragma unroll 4
  for (int64_t k = lane; k < segs; k += 16) top = fmaxf(top, part[k * T + at].x);
  tops[lane][own] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k) top = fmaxf(top, tops[k][own]);
  double s = 0.0;
#pragma unroll 4
  for (int64_t k = lane; k < segs; k += 16) {
    const float2 p = part[k * T + at];
    // (a segment of -inf alone has sum 0, or NaN)
    s += p.x == -INFINITY ? (double)p.y : (double)p.y * exp((double)p.x - (double)top);
  }
  sums[lane][own] = s;
  __syncthreads();
  if (lane != 0 || t >= T) return;
  s = 0.0;
  for (int k = 0; k < 16; ++k) s += sums[k][own];
  finish_token(O, t, top, s, target_z[t]);
}

// A short vocabulary's logits of a token in one workgroup, start to end.
__global__ __launch_bounds__(256) void head_row_kernel(PieceArgs A, TokenOut O) {
  __shared__ float red[4], own;
  __shared__ double sums[4];
  const int64_t t = blockIdx.x, target = A.targets[t];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const float X = A.sum[t];
  auto logits = [&](int64_t i, float* z) {
    const Col4 C = col4(A, i);
    const float4 s = *reinterpret_cast<const float4*>(A.S + t * A.lds + i);
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = i + k < A.m ? fmaf(C.a[k], v[k], fmaf(C.o[k], X, C.b[k])) : -INFINITY;
  };
  if (threadIdx.x == 0) own = __uint_as_float(0x7fc00000u);
  __syncthreads();
  float top = -INFINITY;
  for (int64_t i = threadIdx.x * 4; i < A.m; i += 1024) {
    float z[4];
    logits(i, z);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k == target && i + k < A.m) own = z[k];
      else top = fmaxf(top, z[k]);
    }
  }
  for (int o = 32; o; o >>= 1) top = fmaxf(top, shfl_xor_f(top, o));
  if (lane == 0) red[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float from = top == -INFINITY ? 0.f : top;
  double sum = 0.0;
  for (int64_t i = threadIdx.x * 4; i < A.m; i += 1024) {
    float z[4];
    logits(i, z);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = i + k == target ? 0.f : __builtin_amdgcn_exp2f((z[k] - from) * H_LOG2E);
    sum += (double)((z[0] + z[1]) + (z[2] + z[3]));
  }
  for (int o = 32; o; o >>= 1) sum += shfl_d(sum, lane ^ o);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) finish_token(O, t, top, (sums[0] + sums[1]) + (sums[2] + sums[3]), own);
}

__device__ __forceinline__ float dz_factor(const PieceArgs& A, int64_t i) {
  return A.refs ? pow2(-pow2_shift(A.refs[i])) : A.a ? A.a[i] : 1.f;
}

// The largest factor of dz over all rows, in 64 parts.
__global__ __launch_bounds__(256) void head_factor_kernel(PieceArgs A, float* __restrict__ out) {
  __shared__ float red[4];
  float top = 0.f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < A.m; i += 64 * 256) top = bits_max(top, dz_factor(A, i));
  for (int o = 32; o; o >>= 1) top = bits_max(top, shfl_xor_f(top, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = bits_max(bits_max(red[0], red[1]), bits_max(red[2], red[3]));
}

// What a row's dz over all tokens, times the inverse of the tokens' factors, is at most: dz^T's
// operand of each row of the head carries a power of two of its own, so that the gradient of a
// row that no token makes likely is as exact as any other's (under one power of two for all
// rows a row 20 nats below the likeliest kept 11 bits, one 27 nats below none).  509 x 50257:
// 24 us for 102 MB, 4.3 TB/s, the waves waiting 60 % of their time; with the factors that the
// contraction reads per row, whole calls 876 -> 914 us, so.  By its logarithm; a workgroup takes 256 rows and its share of the tokens, a wave every sixteenth of
// those (several shares: `out` is zeroed before, and the largest stays).
constexpr int BOUND_ROWS = 256, BOUND_WAVES = 16;
__global__ __launch_bounds__(64 * BOUND_WAVES) void head_bound_kernel(PieceArgs A, uint32_t* __restrict__ out) {
  __shared__ float red[BOUND_WAVES][BOUND_ROWS];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t i = (int64_t)blockIdx.x * BOUND_ROWS + lane * 4;
  const Col4 C = col4(A, i);
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 4
  for (int64_t t = (int64_t)blockIdx.y * BOUND_WAVES + wave; t < A.t; t += (int64_t)gridDim.y * BOUND_WAVES) {
    const float f = pow2(-pow2_shift(A.xmax[t]));
    // (0: -inf, or NaN, which a maximum passes over)
    const float others = __builtin_amdgcn_logf(fabsf(A.row_scale[t]) * f) - A.row_top[t] * H_LOG2E;
    const float own = __builtin_amdgcn_logf(fabsf(A.row_target[t]) * f);
    const int64_t target = (int64_t)A.targets[t] - A.row0;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < A.m) s = *reinterpret_cast<const float4*>(A.S + t * A.lds + i);
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], i + q == target ? own : fmaf(v[q] + C.b[q], H_LOG2E, others));
  }
  *reinterpret_cast<float4*>(&red[wave][lane * 4]) = make_float4(top[0], top[1], top[2], top[3]);
  __syncthreads();
  if (threadIdx.x >= BOUND_ROWS) return;
  const int64_t row = (int64_t)blockIdx.x * BOUND_ROWS + threadIdx.x;
  float most = -126.f;   // (a factor of 2^126 at most)
#pragma unroll
  for (int w = 0; w < BOUND_WAVES; ++w) most = fmaxf(most, red[w][threadIdx.x]);
  if (row >= A.m) return;
  const uint32_t bits = __float_as_uint(__builtin_amdgcn_exp2f(most));
  if (gridDim.y > 1) atomicMax(out + row, bits);
  else out[row] = bits;
}
hipError_t launch_bound(const PieceArgs& A, uint32_t* out, hipStream_t st) {
  const int64_t groups = (A.m + BOUND_ROWS - 1) / BOUND_ROWS;
  const int64_t shares = std::max<int64_t>(1, std::min(256 / groups, (A.t + 127) / 128));
  if (shares > 1) {
    const hipError_t e = launch_fill_i32(reinterpret_cast<int32_t*>(out), A.m, 0, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(head_bound_kernel, dim3((unsigned)groups, (unsigned)shares), dim3(64 * BOUND_WAVES), 0, st, A, out);
  return hipGetLastError();
}

// A 64 x 64 tile of dz: its planes, its transpose's (turned in LDS: a lane stores four
// tokens of a row), its rows' and columns' sums.  509 x 50257, with the transpose in two
// terms: 72 us for 258 MB, 3.6 TB/s; vector instructions 65 % of the clocks.
__global__ __launch_bounds__(256) void head_grad_kernel(PieceArgs A) {
  __shared__ float tl[64][65];
  __shared__ float cs[3][4][64];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4, wave = wave_id();
  const int64_t tiles = A.mp / 64, t0 = blockIdx.x / tiles * 64, i0 = blockIdx.x % tiles * 64, i = i0 + cx * 4;
  const Col4 C = col4(A, i);
  const float mid = A.mid >= 0 ? A.levels[A.mid] : 0.f, fm = A.d ? largest_factor(A) : 0.f;
  const float off = A.mid == A.centre ? 0.f : A.levels[A.centre];
  float f[4] = {0.f, 0.f, 0.f, 0.f}, od[4], sums[3][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (A.d && i + q < A.m) f[q] = dz_factor(A, i + q);
    od[q] = fmaf(C.a[q], off, C.o[q]);
    sums[0][q] = sums[1][q] = sums[2][q] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t t = t0 + ry + 16 * k;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < A.t && A.weight[t] != 0.f) {
      const float X = A.sum[t], top = A.row_top[t], scale = A.row_scale[t];
      const int64_t target = (int64_t)A.targets[t] - A.row0;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < A.m) s = *reinterpret_cast<const float4*>(A.S + t * A.lds + i);
      const float sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (i + q >= A.m) continue;
        const float z = fmaf(C.a[q], sv[q], fmaf(C.o[q], X, C.b[q]));
        v[q] = i + q == target ? A.row_target[t] : scale == 0.f ? 0.f : __builtin_amdgcn_exp2f((z - top) * H_LOG2E) * scale;
        sums[0][q] += v[q];
        sums[1][q] = fmaf(v[q], fmaf(mid, X, sv[q]), sums[1][q]);
        sums[2][q] = fmaf(v[q], X, sums[2][q]);
      }
      if (A.d) {
        const uint32_t bound = abs_bits(A.row_target[t] * fm);
        if (blockIdx.x % tiles == 0 && cx == 0) A.dmax[t] = bound;
        const float g = pow2(pow2_shift(bound));
        float u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] = i + q == target && A.own_target ? 0.f : A.raw_d ? v[q] : v[q] * f[q] * g;
        put_dz(A, t, i, u);
      }
    } else if (A.d && t < A.t) {
      if (blockIdx.x % tiles == 0 && cx == 0) A.dmax[t] = 0;
      put_dz(A, t, i, v);
    }
    if (A.rowpart) {
      const float s = sum16(fmaf(v[0], od[0], v[1] * od[1]) + fmaf(v[2], od[2], v[3] * od[3]));
      if (cx == 0 && t < A.t) A.rowpart[t * tiles + blockIdx.x % tiles] = s;
    }
    const float ft = A.dt && t < A.t ? pow2(-pow2_shift(A.xmax[t])) : 1.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) tl[ry + 16 * k][cx * 4 + q] = v[q] * ft;
  }
  if (A.colpart || A.dbias) {
#pragma unroll
    for (int c = 0; c < 3; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float s = sums[c][q];
        s += shfl_xor_f(s, 16);
        s += shfl_xor_f(s, 32);
        if ((threadIdx.x & 63) < 16) cs[c][wave][cx * 4 + q] = s;
      }
  }
  __syncthreads();
  if ((A.colpart || A.dbias) && threadIdx.x < 192) {
    const int c = threadIdx.x >> 6, q = threadIdx.x & 63;
    const float sum = (cs[c][0][q] + cs[c][1][q]) + (cs[c][2][q] + cs[c][3][q]);
    float* out = c == 0 ? A.dbias : c == 1 ? A.dscale : A.doffset;
    if (i0 + q < A.m) {
      if (A.colpart) A.colpart[(t0 / 64 * 3 + c) * A.m + i0 + q] = sum;
      else if (out) out[i0 + q] = sum;   // (the only tile of tokens)
    }
  }
  if (!A.dt) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = i0 + ry + 16 * k;
    if (r >= A.m) continue;
    const float g = pow2(pow2_shift(A.tmax[r]));
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = tl[cx * 4 + q][ry + 16 * k] * g;
    put_terms(A.dt + q_at(r, t0 + cx * 4, A.tp), A.plane_t, A.terms_t, v);
  }
}

// Columns' sums, added up in order in float64.
__global__ __launch_bounds__(256) void head_colsum_kernel(const float* __restrict__ part, int64_t ttiles, int64_t m,
                                                          float* __restrict__ dbias, float* __restrict__ dscale,
                                                          float* __restrict__ doffset) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= m) return;
  float* out[3] = {dbias, dscale, doffset};
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    if (!out[c]) continue;
    double s = 0.0;
    for (int64_t k = 0; k < ttiles; ++k) s += (double)part[(k * 3 + c) * m + i];
    out[c][i] = (float)s;
  }
}
// Rows' sums over the pieces so far.
__global__ __launch_bounds__(256) void head_rowsum_kernel(const float* __restrict__ part, int64_t tiles, int64_t T, bool first,
                                                          float* __restrict__ rowadd) {
  const int64_t t = (int64_t)blockIdx.x * 4 + wave_id();
  const int lane = threadIdx.x & 63;
  if (t >= T) return;
  double s = 0.0;
  for (int64_t k = lane; k < tiles; k += 64) s += (double)part[t * tiles + k];
  for (int o = 32; o; o >>= 1) s += shfl_d(s, lane ^ o);
  if (lane == 0) rowadd[t] = (float)((first ? 0.0 : (double)rowadd[t]) + s);
}

// Steps of eight columns (a lane's) of a chunk: 64 sums for the tokens.
constexpr int few_dx_steps(int fmt, int tokens) { return q_steps(fmt) < 8 / tokens ? q_steps(fmt) : 8 / tokens; }
// dx from its sums over the pieces, and the targets' terms -w rest W[r] where dz's operand
// leaves them out: the largest of a token's, they would carry their 16-bit rounding into
// all of its row.
struct TargetTerms {
  bool wanted, packed, rows, vec;   // rows: entries times the scale, less the middle level's (the rows' sums have the rest)
  const void* W; int64_t ldw, V;
  int dtype;
  QLayer L;
  const int32_t* targets;
  const float *weight, *row_target;
};
__device__ __forceinline__ void target_row4(const TargetTerms& R, int64_t r, int64_t j, float* w) {
  if (!R.packed) {
    load4(R.W, r * R.ldw + j, R.dtype, R.vec, (int)min((int64_t)4, R.L.n - j), w);
    return;
  }
  q_entries4(R.L, q_code4(R.L, r, j), j, w);
  const float mid = q_centre(R.L);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t g = r * R.L.G + (R.L.G > 1 ? min(j + q, R.L.n - 1) / R.L.group : 0);
    w[q] = R.rows ? R.L.scale[g] * (w[q] - mid) : fmaf(R.L.scale[g], w[q], R.L.offset ? R.L.offset[g] : 0.f);
  }
}
__global__ __launch_bounds__(256) void head_dx_kernel(const float* __restrict__ acc, int splits, int64_t lda, int64_t T, int64_t n,
                                                      const float* __restrict__ rowadd, TargetTerms R, void* __restrict__ dx,
                                                      int64_t ld, int dtype, bool vec) {
  const int64_t quads = (n + 3) / 4, step = (int64_t)gridDim.x * 256;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < T * quads; k += step) {
    const int64_t t = k / quads, j = (k - t * quads) * 4;
    const bool read = R.weight[t] != 0.f;   // (else zeros, whatever the head holds: no 0 times NaN)
    const float add = rowadd && read ? rowadd[t] : 0.f;
    float v[4] = {add, add, add, add};
#pragma unroll 8
    for (int s = 0; s < splits && read; ++s) {
      const float4 q = *reinterpret_cast<const float4*>(acc + ((int64_t)s * T + t) * lda + j);
      v[0] += q.x;
      v[1] += q.y;
      v[2] += q.z;
      v[3] += q.w;
    }
    if (R.wanted && read && R.targets[t] < R.V) {
      float w[4];
      target_row4(R, R.targets[t], j, w);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = fmaf(R.row_target[t], w[q], v[q]);
    }
    store4(dx, t * ld + j, dtype, vec, (int)min((int64_t)4, n - j), v);
  }
}

// dx of up to four tokens straight from the packed codes, with the sums that a packed head's
// gradients are where one affine has a row: no planes (32 bytes written and read for eight
// codes) and no tile of 128 tokens for one.  A lane decodes its row's part of a chunk of columns
// (SP steps of eight; the more tokens, the fewer) and adds dz a times it to columns of its own;
// sixteen rows, a workgroup's waves and the splits of the rows are joined after that alone.
template <int FMT, int TN, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void head_few_dx_kernel(PieceArgs A, QLayer L, bool sums, int splits,
                                                                 float* __restrict__ out, int64_t lda) {
  extern __shared__ __attribute__((aligned(16))) uint32_t few_lds[];
  constexpr int STEPS = q_steps(FMT), SP = few_dx_steps(FMT, TN), PARTS = STEPS / SP, COLS = SP * 32;
  const int lane = threadIdx.x & 63, wave = wave_id(), kb = lane >> 4;
  q_lut_fill<FMT, OpF16>(L, few_lds, 64 * WAVES);
  if (FMT == QF_E8) q_lut_wait<0>();
  __syncthreads();
  const int split = (int)(blockIdx.x % splits), place = (int)(blockIdx.x / splits), c = place / PARTS, part = place % PARTS;
  const int g = L.G > 1 ? (int)((int64_t)c * (STEPS * 32) / L.group) : 0;
  const float mid = q_centre(L), zmid = A.mid >= 0 ? A.levels[A.mid] : 0.f;
  float top[TN], scale[TN], own[TN], X[TN], rest[TN], acc[SP * 8][TN];
  int target[TN];
  bool read[TN];   // (a token that is not has no s)
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const bool live = read[t] = t < A.t && A.weight[min((int64_t)t, A.t - 1)] != 0.f;
    top[t] = live ? A.row_top[t] : 0.f;
    scale[t] = live ? A.row_scale[t] : 0.f;
    own[t] = live ? A.row_target[t] : 0.f;
    X[t] = live ? A.sum[t] : 0.f;
    target[t] = live ? A.targets[t] : -1;
    rest[t] = 0.f;
#pragma unroll
    for (int k = 0; k < SP * 8; ++k) acc[k][t] = 0.f;
  }
  for (int tile = split * WAVES + wave; tile < L.tiles; tile += splits * WAVES) {
    const uint4 code = L.packed[((size_t)tile * L.chunks + c) * 64 + lane];
    const int64_t v = (int64_t)tile * 16 + (lane & 15), at = min(v, A.m - 1);
    const bool live = v < A.m;
    const float a = L.scale[at * L.G + g], o = fmaf(a, mid, L.offset ? L.offset[at * L.G + g] : 0.f);
    const float za = A.a ? A.a[at] : 1.f, zo = A.a ? fmaf(za, zmid, A.o ? A.o[at] : 0.f) : 0.f, zb = A.b ? A.b[at] : 0.f;
    float u[TN], part3[3][4] = {};
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const float s = A.S[min((int64_t)t, A.t - 1) * A.lds + at], z = fmaf(za, s, fmaf(zo, X[t], zb));
      float d = target[t] == v ? own[t] : scale[t] == 0.f ? 0.f : __builtin_amdgcn_exp2f((z - top[t]) * H_LOG2E) * scale[t];
      if (!live) d = 0.f;
      u[t] = d * a;
      rest[t] = fmaf(d, o, rest[t]);
      part3[0][t] = d;
      part3[1][t] = read[t] ? fmaf(d, fmaf(zmid, X[t], s), 0.f) : 0.f;   // (rounded here: no product joins a sum)
      part3[2][t] = fmaf(d, X[t], 0.f);
    }
    if (sums && place == 0 && kb == 0 && live) {   // (in head_grad_kernel's order)
      float* const to[3] = {A.dbias, A.dscale, A.doffset};
#pragma unroll
      for (int k = 0; k < 3; ++k) to[k][v] = (part3[k][0] + part3[k][1]) + (part3[k][2] + part3[k][3]);
    }
    uint4 w = code;
    if constexpr (PARTS == 2) w = part ? make_uint4(code.z, code.w, 0, 0) : make_uint4(code.x, code.y, 0, 0);
    if constexpr (PARTS == 4) w = make_uint4(part == 0 ? code.x : part == 1 ? code.y : part == 2 ? code.z : code.w, 0, 0, 0);
#pragma unroll
    for (int s = 0; s < SP; ++s) {
      const v4u e = q_decode<FMT, OpF16>(L, few_lds, w, s);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float x = OpF16::val(q & 1 ? e[q >> 1] >> 16 : e[q >> 1]);
#pragma unroll
        for (int t = 0; t < TN; ++t) acc[s * 8 + q][t] = fmaf(x, u[t], acc[s * 8 + q][t]);
      }
    }
  }
  __syncthreads();   // (the table's place takes the sums)
  float* red = reinterpret_cast<float*>(few_lds);   // [WAVES][TN][COLS]
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const float r = sum16(rest[t]);
#pragma unroll
    for (int k = 0; k < SP * 8; ++k) {
      const float s = sum16(acc[k][t]) + r;
      if ((lane & 15) == (k & 15)) red[(wave * TN + t) * COLS + ((k >> 3) * 4 + kb) * 8 + (k & 7)] = s;
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < TN * COLS; k += 64 * WAVES) {
    const int t = k / COLS, q = k % COLS;
    const int64_t j = ((int64_t)c * STEPS + part * SP) * 32 + q;
    if (t >= A.t || j >= lda) continue;
    float s = 0.f;
    for (int w = 0; w < WAVES; ++w) s += red[(w * TN + t) * COLS + q];
    out[((int64_t)split * A.t + t) * lda + j] = s;
  }
}
struct FewDx {
  int tokens, waves, splits;
  unsigned grid;
  size_t shared;
};
FewDx few_dx_plan(const QLayer& L, int64_t T) {
  FewDx P;
  P.tokens = T <= 1 ? 1 : T <= 2 ? 2 : 4;
  // (E8's table fills a CU's LDS)
  P.waves = L.fmt == QF_E8 ? 16 : 4;
  const int steps = few_dx_steps(L.fmt, P.tokens);
  const int64_t places = (int64_t)L.chunks * (q_steps(L.fmt) / steps), most = L.fmt == QF_E8 ? 256 : 1024;
  P.splits = (int)std::max<int64_t>(1, std::min({most / places, (L.tiles + P.waves - 1) / (int64_t)P.waves, (int64_t)64}));
  P.grid = (unsigned)(places * P.splits);
  P.shared = std::max((size_t)q_lut_words(L.fmt, (L.lut_entries + 3) / 4 * 4) * 4, (size_t)P.waves * P.tokens * steps * 32 * 4);
  return P;
}
template <int FMT, int WAVES>
hipError_t launch_few_dx(const FewDx& P, const PieceArgs& A, const QLayer& L, bool sums, float* out, int64_t lda, hipStream_t st) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(P.grid), dim3(64 * WAVES), P.shared, st, A, L, sums, P.splits, out, lda);
    return hipGetLastError();
  };
  return P.tokens == 1   ? go(head_few_dx_kernel<FMT, 1, WAVES>)
         : P.tokens == 2 ? go(head_few_dx_kernel<FMT, 2, WAVES>)
                         : go(head_few_dx_kernel<FMT, 4, WAVES>);
}

bool whole_quads(const void* p, int64_t ld, int dtype) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (dtype == DT_F32 ? 16 : 8) == 0 && ld % 4 == 0);
}

// Rows row0 .. row0 + rows - 1 of a packed layer (row0 a multiple of 16).
QLayer layer_rows(const QLayer& L, int64_t row0, int64_t rows) {
  QLayer P = L;
  P.m = rows;
  P.tiles = (int)((rows + 15) / 16);
  if (L.packed) P.packed = L.packed + (size_t)(row0 / 16) * L.chunks * 64;
  if (L.scale) P.scale = L.scale + row0 * L.G;
  if (L.offset) P.offset = L.offset + row0 * L.G;
  return P;
}

#define H_TRY(x)                            \
  do {                                      \
    const hipError_t e_ = (x);              \
    if (e_ != hipSuccess) return e_;        \
  } while (0)
#define H_LAUNCH(kernel, grid, block, ...)                                            \
  do {                                                                                \
    hipLaunchKernelGGL(kernel, dim3 grid, dim3(block), 0, st, __VA_ARGS__);           \
    H_TRY(hipGetLastError());                                                         \
  } while (0)

hipError_t head(const HeadArgs& A, char* base, size_t* bytes, hipStream_t st) {
  const QLayer& L = A.L;
  const int64_t T = A.t, V = L.m, n = L.n, Kp = up64(n), tp = up64(T), ttiles = tp / 64;
  const bool f32 = A.dtype == DT_F32, weights = A.dense || L.G > 1;   // the planes hold weights, not entries
  const int XP = f32 ? 2 : 1;
  // A matrix in 16 bits is one term, exact; a group's a e + o takes two, as float32 does.
  const int WP = A.dense && !f32 ? 1 : weights ? 2 : 1;
  const bool grads = A.need_dx || A.need_dhead, product = A.need_dhead && weights;
  // A 16-bit matrix whose rows the product's tiles can read in place goes without planes.
  const bool in_place = A.dense && !f32 && n % 64 == 0 && A.ldw % 8 == 0 && A.ldw <= (1 << 20) &&
                        reinterpret_cast<uintptr_t>(A.W) % 16 == 0;
  const int DX = f32 ? 2 : 1;                   // dz for dx
  const int WX = f32 ? WP : 1;                  // the weights for dx: as many terms as dz
  // dz^T for dW: one term has eight times a bfloat16 result's precision, and no more than a float16 one's.
  const int DT = A.dense && A.dtype == DT_BF16 ? 1 : 2;
  const bool contract = !A.dense && L.group % Q_CONTRACT == 0;
  // Logits that fit half of the last-level cache are kept for the gradients: written and
  // read there, they cost less than their product.  Others leave the product as
  // statistics, and as dz.
  const int64_t lds = (V + 255) / 256 * 256;
  const bool kept = T * lds * 4 <= H_BYTES;
  // rows of a piece
  int64_t rows = (kept ? H_PLANES : H_PIECE) / (WP * Kp * 2);
  if (!kept) rows = std::min(rows, H_PIECE / (T * 4));
  rows = std::min(std::max(rows / 256 * 256, H_ROWS), lds);
  // (a wave per group of a row sums up a dW in memory: fewer than 2^32 threads; whatever is wanted,
  // as the workspace is sized)
  if (!A.dense && !contract) rows = std::min(rows, (((int64_t)1 << 26) - 1) / L.G / 256 * 256);
  const int64_t pieces = (V + rows - 1) / rows;
  const HeadTile tile = head_tile(rows, T);
  // The gradients' pass takes logits in memory: those that are kept, or a piece's, formed again
  // there where dz^T is wanted (a row's factor is known once all its tokens' dz are).
  const bool stored = kept || product;
  // Few tokens: straight from the packed codes.
  const bool few = kept && !A.dense && q_few_rows(L, A.dtype, T);
  // ... and their input gradient (planes_dx: through planes).
  const bool few_dx = few && A.need_dx && T <= H_FEW, planes_dx = A.need_dx && !few_dx;
  // (A token of 32000 logits: 32 segments of 1024, with their join 10 us; 8 of 4096 would leave
  // most CUs without one.  Many tokens: 509 x 50257, 4096 rows a workgroup 32 us.)
  const int64_t seg_rows = T <= 64 ? 1024 : 4096;
  // One workgroup a token, start to end. (Longer rows in segments: a token of 32000 logits takes
  // 15.6 us in one workgroup of sixteen waves, 8 in segments with their join.)
  const bool short_rows = kept && V <= 16384;
  const int64_t seg = kept ? seg_rows : tile.rows, all_segs = (V + seg - 1) / seg;
  const int64_t row_tiles = stored ? rows / 64 : rows / tile.rows, token_tiles = stored ? ttiles : (T + 127) / 128;
  Carve W{base};
  TokenArgs K;
  memset(&K, 0, sizeof(K));
  K.weight = W.take<float>((size_t)T * 4);
  K.sum = W.take<float>((size_t)T * 4);
  K.target_z = W.take<float>((size_t)T * 4);
  K.rowmax = W.take<uint32_t>((size_t)T * 4);
  float* fpart = W.take<float>(64 * 4);
  float* ones = W.take<float>(!A.dense && !weights ? (size_t)V * 4 : 0);
  float* row_top = W.take<float>((size_t)T * 4);
  float* row_scale = W.take<float>((size_t)T * 4);
  float* row_target = W.take<float>((size_t)T * 4);
  const int64_t Kx = few ? (int64_t)L.chunks * q_chunk(L.fmt) : Kp;
  K.plane = up16(T) * Kx;
  K.planes = W.take<uint16_t>((size_t)XP * K.plane * 2);
  uint32_t* refs = W.take<uint32_t>(weights ? (size_t)V * 4 : 0);
  // (as many tokens as come straight from the codes both ways lay no plane out, whatever is wanted)
  const bool planes = !few || T > H_FEW;
  uint16_t* wp = W.take<uint16_t>(planes ? (size_t)WP * up16(rows) * Kp * 2 : 0);
  const int64_t lds_p = kept ? lds : rows;   // of the logits that the gradients' pass takes
  float* S = W.take<float>(stored ? (size_t)T * lds_p * 4 : 0);
  float2* part = W.take<float2>((size_t)all_segs * T * sizeof(float2));
  QGemm gz, gx, gw;
  memset(&gz, 0, sizeof(gz));
  memset(&gx, 0, sizeof(gx));
  memset(&gw, 0, sizeof(gw));
  q_pairs(gz, WP, XP);
  q_pairs(gx, WX, DX);
  q_pairs(gw, XP, DT);
  size_t ps = 0;
  auto both_sizes = [&](auto f) {   // a whole piece's, and the last's
    f(std::min(rows, V));
    f(V - (pieces - 1) * rows);
  };
  if (stored && !few) both_sizes([&](int64_t nr) { ps = std::max(ps, q_gemm_workspace(nr, T, Kp, gz.npairs)); });
  uint16_t *d = nullptr, *dt = nullptr;
  uint32_t *dmax = nullptr, *tmax = nullptr;
  float *rowpart = nullptr, *rowadd = nullptr, *acc = nullptr, *colpart = nullptr, *dW = nullptr;
  float2* cpart = nullptr;
  const int64_t lda = (n + 3) / 4 * 4, cblocks = (n + Q_CONTRACT - 1) / Q_CONTRACT;
  int splits = 1, dx_splits = 1;
  // (workspaces are sized without the offset's pointer: room for its sums either way)
  const bool sums = planes_dx && !weights && L.has_offset();
  if (few_dx) {
    dx_splits = few_dx_plan(L, T).splits;
    acc = W.take<float>((size_t)dx_splits * T * lda * 4);
  }
  if (planes_dx) {
    d = W.take<uint16_t>((size_t)DX * up16(T) * rows * 2);
    dmax = W.take<uint32_t>((size_t)T * 4);
    rowpart = W.take<float>((size_t)T * row_tiles * 4);
    rowadd = W.take<float>((size_t)T * 4);
    dx_splits = head_dx_splits(n, T, rows, gx.npairs);
    acc = W.take<float>((size_t)dx_splits * T * lda * 4);
  }
  if (A.need_dhead) colpart = W.take<float>((size_t)token_tiles * 3 * rows * 4);
  if (product) {
    K.plane_again = up16(T) * Kp;
    K.Kp_again = Kp;
    K.again = W.take<uint16_t>((size_t)XP * K.plane_again * 2);
    dt = W.take<uint16_t>((size_t)DT * up16(rows) * tp * 2);
    tmax = W.take<uint32_t>((size_t)rows * 4);
    if (contract) {
      both_sizes([&](int64_t nr) { splits = std::max(splits, q_gemm_splits(n, nr, tp, gw.npairs)); });
      cpart = W.take<float2>((size_t)splits * rows * cblocks * sizeof(float2));
    } else {
      if (!A.dense) dW = W.take<float>((size_t)rows * lda * 4);
      both_sizes([&](int64_t nr) { ps = std::max(ps, q_gemm_workspace(n, nr, tp, gw.npairs)); });
    }
  }
  float* gpart = W.take<float>(ps);
  if (bytes) *bytes = W.at;
  if (!base) return hipSuccess;

  // the tokens
  K.x = A.x; K.ldx = A.ldx;
  K.dtype = A.dtype;
  K.t = T; K.n = n; K.V = V;
  K.targets = A.targets;
  K.weights = A.weights;
  K.vec = whole_quads(A.x, A.ldx, A.dtype);
  K.terms = XP;
  K.Kp = Kx;
  K.frags = few;
  K.raw = in_place && A.dtype == DT_BF16;
  const bool twice = product && (K.raw || few);   // the logits' operand is no float16 one in operand order
  const uint16_t* xplanes = twice ? K.again : K.planes;
  const int64_t xplane = twice ? K.plane_again : K.plane;
  if (!twice) K.again = nullptr;
  K.ones = few && !weights ? ones : nullptr;
  if (planes_dx && !weights) {
    K.scale = L.scale;
    K.fpart = fpart;
  }
  const uint32_t* rowmax = K.raw ? nullptr : K.rowmax;
  H_LAUNCH(head_token_kernel, ((unsigned)(up16(T) + (K.fpart ? 64 : 0) + (K.ones ? (V + 255) / 256 : 0))), 256, K);
  PieceArgs P;
  memset(&P, 0, sizeof(P));
  P.lds = lds_p;
  P.t = T;
  P.weight = K.weight; P.sum = K.sum;
  P.targets = A.targets;
  P.target_z = K.target_z;
  P.row_top = row_top; P.row_scale = row_scale; P.row_target = row_target;
  P.tmax = tmax; P.xmax = K.rowmax;
  P.fmax = in_place ? nullptr : fpart;
  P.dmax = dmax;
  P.terms_d = DX; P.terms_t = DT;
  P.tp = tp;
  P.levels = L.levels;
  P.centre = !weights && (L.fmt == QF_NIB || L.fmt == QF_BYTE) ? L.K / 2 : -1;
  P.mid = few ? -1 : P.centre;
  QLayer Q;
  // The piece's rows, and its planes.
  auto piece = [&](int64_t k, bool planes, int terms) -> hipError_t {
    const int64_t r0 = k * rows, nr = std::min(rows, V - r0), plane = up16(nr) * Kp;
    Q = layer_rows(L, r0, nr);
    P.m = nr;
    P.row0 = r0;
    P.mp = up64(nr);
    P.plane_d = up16(T) * P.mp;
    P.plane_t = up16(nr) * tp;
    P.S = kept ? S + r0 : S;
    P.a = weights ? nullptr : Q.scale;
    P.o = weights ? nullptr : Q.offset;
    P.b = A.bias ? A.bias + r0 : nullptr;
    P.refs = weights && !in_place ? refs + r0 : nullptr;
    P.part = part + r0 / tile.rows * T;   // (pieces begin at multiples of the tile's rows)
    if (planes && A.dense && !in_place) {
      DenseArgs D;
      memset(&D, 0, sizeof(D));
      D.W = static_cast<const char*>(A.W) + r0 * A.ldw * (f32 ? 4 : 2);
      D.ldw = A.ldw;
      D.dtype = A.dtype;
      D.vec = whole_quads(D.W, D.ldw, A.dtype);
      D.m = nr; D.n = n; D.Kp = Kp;
      D.terms = WP;
      D.refs = refs + r0;
      D.out = wp; D.plane = plane;
      H_LAUNCH(head_dense_kernel, ((unsigned)(up16(nr) / 4)), 256, D);
    } else if (planes && !A.dense) {
      if (weights) H_TRY(launch_q_bounds(Q, refs + r0, st));
      H_TRY(launch_q_unpack(Q, Kp, weights ? terms : 0, refs + r0, wp, plane, st));
    }
    gz.A = wp; gz.planeA = plane;
    if (in_place) {
      gz.A = reinterpret_cast<const uint16_t*>(static_cast<const char*>(A.W) + r0 * A.ldw * 2);
      gz.lda = A.ldw;
      gz.bf16 = A.dtype == DT_BF16;
    }
    gz.B = K.planes; gz.planeB = K.plane;
    gz.M = nr; gz.N = T; gz.K = Kp;
    return hipSuccess;
  };
  if (few) {
    QLayer F = L;
    if (!weights) {
      F.scale = ones;
      F.offset = nullptr;
    }
    QOut O;
    memset(&O, 0, sizeof(O));
    O.y = S; O.ldy = lds;
    O.rowmax = rowmax;
    O.mid = -1;
    O.dtype = DT_F32;
    O.vec = 1;
    O.rows = T; O.cols = V;
    H_TRY(launch_q_skinny(F, K.planes, 0, K.plane, T, XP, false, O, st));
  }
  auto store = [&]() {   // the piece's logits, as P.S says
    gz.O.y = const_cast<float*>(P.S); gz.O.ldy = lds_p;
    gz.O.rowmax = rowmax;
    gz.O.colmax = P.refs;
    gz.O.mid = -1;
    gz.O.dtype = DT_F32;
    gz.O.vec = 1;
    gz.O.rows = T; gz.O.cols = P.m;
    return launch_q_gemm(gz, gpart, st);
  };
  for (int64_t k = 0; k < pieces && !few; ++k) {
    H_TRY(piece(k, true, WP));
    H_TRY(kept ? store() : launch_head_gemm(gz, P, rowmax, false, st));
  }
  const TokenOut O = {K.weight, A.loss, row_top, row_scale, row_target};
  if (kept) {
    PieceArgs F = P;   // all of it
    F.m = V;
    F.row0 = 0;
    F.S = S;
    F.a = weights ? nullptr : L.scale;
    F.o = weights ? nullptr : L.offset;
    F.b = A.bias;
    F.part = part;
    if (short_rows) H_LAUNCH(head_row_kernel, ((unsigned)T), 256, F, O);
    else if (seg == 1024) H_LAUNCH(head_stats_kernel<1>, ((unsigned)T, (unsigned)all_segs), 256, F);
    else H_LAUNCH(head_stats_kernel<4>, ((unsigned)T, (unsigned)all_segs), 256, F);
  }
  if (!short_rows) H_LAUNCH(head_join_kernel, ((unsigned)((T + 15) / 16)), 256, part, all_segs, T, K.target_z, O);
  if (!grads) return hipSuccess;
  P.raw_d = K.raw;
  P.own_target = planes_dx && !f32 && (P.raw_d || A.dtype == DT_F16);
  if (planes_dx && weights && !in_place) {
    PieceArgs F = P;
    F.m = V;
    F.refs = refs;
    if (few) H_TRY(launch_q_bounds(L, refs, st));
    H_LAUNCH(head_factor_kernel, (64), 256, F, fpart);
  }
  if (few_dx) {
    PieceArgs F = P;
    F.m = V;
    F.S = S;
    F.a = weights ? nullptr : L.scale;
    F.o = weights ? nullptr : L.offset;
    F.b = A.bias;
    F.dbias = A.dbias; F.dscale = A.dscale; F.doffset = A.doffset;
    const bool own_sums = A.need_dhead && !weights;
    const FewDx D = few_dx_plan(L, T);
    H_TRY(L.fmt == QF_E8     ? (launch_few_dx<QF_E8, 16>(D, F, L, own_sums, acc, lda, st))
          : L.fmt == QF_NIB  ? (launch_few_dx<QF_NIB, 4>(D, F, L, own_sums, acc, lda, st))
          : L.fmt == QF_BYTE ? (launch_few_dx<QF_BYTE, 4>(D, F, L, own_sums, acc, lda, st))
                             : (launch_few_dx<QF_VEC, 4>(D, F, L, own_sums, acc, lda, st)));
  }
  // (a single piece's planes are still there)
  const bool again = pieces > 1 || few, rest = planes_dx || product || (A.need_dhead && !few_dx);
  for (int64_t k = 0; k < pieces && rest; ++k) {
    H_TRY(piece(k, again && (!kept || planes_dx), kept ? WX : WP));   // (kept: for dx alone)
    const int64_t r0 = P.row0, nr = P.m, mp = P.mp;
    P.d = planes_dx ? d : nullptr;
    P.rowpart = sums ? rowpart : nullptr;
    P.dt = product ? dt : nullptr;
    const bool straight = stored && ttiles == 1;   // no tiles of tokens to add up
    P.colpart = A.need_dhead && !straight ? colpart : nullptr;
    if (A.need_dhead && straight) {
      P.dbias = A.dbias + r0;
      P.dscale = weights ? nullptr : A.dscale + r0;
      P.doffset = weights ? nullptr : A.doffset + r0;
    }
    if (!kept && product) H_TRY(store());
    if (product) H_TRY(launch_bound(P, tmax, st));
    if (stored)
      H_LAUNCH(head_grad_kernel, ((unsigned)(mp / 64 * ttiles)), 256, P);
    else
      H_TRY(launch_head_gemm(gz, P, rowmax, true, st));
    const HeadTile own = head_tile(nr, T);   // (of the last piece, smaller)
    if (P.colpart)
      H_LAUNCH(head_colsum_kernel, ((unsigned)((nr + 255) / 256)), 256, colpart,
               stored ? ttiles : (T + own.tokens - 1) / own.tokens, nr, A.dbias + r0,
               weights ? nullptr : A.dscale + r0, weights ? nullptr : A.doffset + r0);
    if (sums) H_LAUNCH(head_rowsum_kernel, ((unsigned)((T + 3) / 4)), 256, rowpart,
                       stored ? mp / 64 : (nr + own.rows - 1) / own.rows, T, k == 0, rowadd);
    if (planes_dx) {
      gx.A = gz.A; gx.lda = gz.lda; gx.planeA = gz.planeA;
      gx.bf16 = gz.bf16;
      gx.acols = Kp; gx.arows = nr;
      gx.B = d; gx.planeB = P.plane_d;
      gx.M = n; gx.N = T; gx.K = mp;
      H_TRY(launch_head_dx(gx, P.raw_d ? nullptr : dmax, acc, lda, rows, k == 0, st));
    }
    if (product) {
      gw.A = xplanes; gw.planeA = xplane;
      gw.acols = Kp; gw.arows = T;
      gw.B = dt; gw.planeB = P.plane_t;
      gw.M = n; gw.N = nr; gw.K = tp;
      gw.O.rowmax = tmax;
      gw.O.mid = -1;
      gw.O.rows = nr; gw.O.cols = n;
      if (A.dense) {
        gw.O.y = static_cast<char*>(A.dW) + r0 * A.lddw * (f32 ? 4 : 2); gw.O.ldy = A.lddw;
        gw.O.dtype = A.dtype;
        gw.O.vec = whole_quads(gw.O.y, A.lddw, A.dtype);
        H_TRY(launch_q_gemm(gw, gpart, st));
      } else {
        gw.O.y = dW; gw.O.ldy = lda;
        gw.O.dtype = DT_F32;
        gw.O.vec = 1;
        gw.L = Q;
        gw.cpart = contract ? cpart : nullptr;
        gw.cblocks = cblocks;
        H_TRY(launch_q_gemm(gw, gpart, st));
        H_TRY(launch_q_affine_sums(Q, contract ? cpart : nullptr, q_gemm_splits(n, nr, tp, gw.npairs), cblocks, dW, lda,
                                   A.dscale + r0 * L.G, A.doffset + r0 * L.G, st));
      }
    }
  }
  TargetTerms R;
  memset(&R, 0, sizeof(R));
  R.wanted = P.own_target;
  R.packed = !A.dense; R.rows = !weights;
  R.vec = whole_quads(A.W, A.ldw, A.dtype);
  R.W = A.W; R.ldw = A.ldw; R.V = V;
  R.dtype = A.dtype;
  R.L = L;
  R.targets = A.targets; R.weight = K.weight; R.row_target = row_target;
  if (A.need_dx)
    H_LAUNCH(head_dx_kernel, ((unsigned)std::min<int64_t>((T * (lda / 4) + 255) / 256, 4096)), 256, acc, dx_splits, lda, T, n,
             sums ? rowadd : nullptr, R, A.dx, A.lddx, A.dtype, whole_quads(A.dx, A.lddx, A.dtype));
  return hipSuccess;
}

}  // namespace

size_t head_workspace(const HeadArgs& A) {
  size_t b = 0;
  (void)head(A, nullptr, &b, nullptr);
  return b;
}
hipError_t launch_head(const HeadArgs& A, void* ws, hipStream_t st) {
  return head(A, static_cast<char*>(ws), nullptr, st);
}

}  // namespace mpq
