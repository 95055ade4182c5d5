// A head's logits out of the product's registers: their statistics, or dz with its
// sums and operand planes (head.hip has the mathematics).
//
// The product is qgemm.hip's; a lane ends with four consecutive rows of the head for
// one token in each of its subtiles, and what it needs of a row (scale, offset, bias)
// comes from LDS, of a token from registers.  The statistics are a maximum and a
// sum of exponentials over the lane's rows, then over the four lanes and the waves that
// share a token: 8 bytes a token and tile leave.  dz leaves as operand planes
// (16 bits a logit and term) and as sums over the tile's tokens and rows.
//
// Bound.  As the product alone: 2048 tokens, 32768 rows of 4096 columns, statistics 380 us
// (1.45 PFLOP/s; products alone reach 2.07), dz 445 (for a packed head with an affine per row,
// or for dx alone).  The matrix cores are busy 66 % of the clocks (55 % with dz), which their
// power holds at 1.97 GHz; without any load or LDS read in the loop the statistics would still
// take 330.  What is left is the step's barrier and the
// epilogue (some 12 vector instructions a logit for the statistics, 35 for dz) in the one
// workgroup that fits a CU.  Tried: four waves of 128 x 128 each, statistics 440 us; two
// workgroups of 256 x 128 on a CU 408, dz 468.
#include <algorithm>
#include "qgemm_tile.h"
#include "head.h"

namespace mpq {

namespace {

template <typename T, int BM, int BN, int WM, int WN, bool GRADS, int AMODE>
__global__ __launch_bounds__(64 * WM * WN, 2) void head_gemm_kernel(QGemm g, PieceArgs A, const uint32_t* __restrict__ rowmax) {
  constexpr int SM = BM / WM / 16, SN = BN / WN / 16;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[gemm_stages(BM, BN)][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, kb = lane >> 4;
  int split;
  int64_t i0, j0;
  v4f acc[SM][SN];
  q_gemm_tile<T, BM, BN, WM, WN, AMODE>(g, 1, lds, acc, split, i0, j0);
  // The rows of the head: factor of s, of X, what is added; dz's factor.
  float* const cols = reinterpret_cast<float*>(lds);
  float *ca = cols, *co = cols + BM, *cb = cols + 2 * BM, *cf = cols + 3 * BM, *work = cols + 4 * BM;
  const float mid = A.mid >= 0 ? A.levels[A.mid] : 0.f;
  for (int k = threadIdx.x; k < BM; k += 64 * WM * WN) {
    const int64_t i = i0 + k;
    float a = 0.f, o = 0.f, b = -INFINITY, f = 0.f;   // no row: a logit of -inf
    if (i < A.m) {
      a = A.a ? A.a[i] : 1.f;
      o = A.a ? fmaf(a, mid, A.o ? A.o[i] : 0.f) : 0.f;
      b = A.b ? A.b[i] : 0.f;
      f = a;
      if (A.refs) {
        f = pow2(-pow2_shift(A.refs[i]));
        if (AMODE == A_BLOCKS) a = f;   // (rows read in place are what they are)
      }
    }
    ca[k] = a;
    co[k] = o;
    cb[k] = b;
    cf[k] = f;
  }
  __syncthreads();
  const int at = wm * SM * 16 + 4 * kb;   // this lane's first row in the tile, and every 16 from there
  if constexpr (!GRADS) {
    float2* red = reinterpret_cast<float2*>(work);   // [WM][BN]
#pragma unroll
    for (int jj = 0; jj < SN; ++jj) {
      const int jt = (wn * SN + jj) * 16 + r;
      const int64_t t = min(j0 + jt, A.t - 1);
      const float f = rowmax ? pow2(-pow2_shift(rowmax[t])) : 1.f, X = A.sum[t];
      const int64_t target = (int64_t)A.targets[t] - A.row0 - i0 - at;
      float top = -INFINITY, own = 0.f;
      bool here = false;
#pragma unroll
      for (int s = 0; s < SM; ++s) {
        const v4f a = *reinterpret_cast<const v4f*>(ca + at + s * 16), o = *reinterpret_cast<const v4f*>(co + at + s * 16),
                  b = *reinterpret_cast<const v4f*>(cb + at + s * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float z = fmaf(a[k], acc[s][jj][k] * f, fmaf(o[k], X, b[k]));
          if (target == s * 16 + k) {
            own = z;
            here = true;
            z = -INFINITY;
          }
          acc[s][jj][k] = z;
          top = fmaxf(top, z);
        }
      }
      if (here && j0 + jt < A.t && i0 + at + target < A.m) A.target_z[t] = own;
      top = fmaxf(top, shfl_xor_f(top, 16));
      top = fmaxf(top, shfl_xor_f(top, 32));
      const float from = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < SM; ++s) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = __builtin_amdgcn_exp2f((acc[s][jj][k] - from) * H_LOG2E);
        sum += (e[0] + e[1]) + (e[2] + e[3]);
      }
      sum += shfl_xor_f(sum, 16);
      sum += shfl_xor_f(sum, 32);
      if (kb == 0) red[wm * BN + jt] = make_float2(top, sum);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < BN; k += 64 * WM * WN) {
      if (j0 + k >= A.t) continue;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WM; ++w) top = fmaxf(top, red[w * BN + k].x);
#pragma unroll
      for (int w = 0; w < WM; ++w) {
        const float2 p = red[w * BN + k];
        sum += p.x == -INFINITY ? p.y : p.y * __builtin_amdgcn_exp2f((p.x - top) * H_LOG2E);
      }
      A.part[i0 / BM * A.t + j0 + k] = make_float2(top, sum);
    }
  } else {
    float f[SN], X[SN], top[SN], scale[SN], own[SN], gd[SN], rows[SN];
    int target[SN];
    const float fm = A.d ? largest_factor(A) : 0.f;
#pragma unroll
    for (int jj = 0; jj < SN; ++jj) {
      const int64_t t = j0 + (wn * SN + jj) * 16 + r, th = min(t, A.t - 1);
      const bool live = t < A.t;
      f[jj] = rowmax ? pow2(-pow2_shift(rowmax[th])) : 1.f;
      X[jj] = A.sum[th];
      top[jj] = A.row_top[th];
      scale[jj] = live ? A.row_scale[th] : 0.f;
      own[jj] = live ? A.row_target[th] : 0.f;
      const int64_t d = (int64_t)A.targets[th] - A.row0 - i0 - at;
      target[jj] = d >= 0 && d < SM * 16 ? (int)d : -1;
      const uint32_t bound = abs_bits(own[jj] * fm);
      if (A.d && i0 == 0 && wm == 0 && kb == 0 && live) A.dmax[t] = bound;
      gd[jj] = pow2(pow2_shift(bound));
      rows[jj] = 0.f;
    }
    float* red = work;   // [WN][3][BM], and [WM][BN] after it
#pragma unroll
    for (int s = 0; s < SM; ++s) {
      const v4f a = *reinterpret_cast<const v4f*>(ca + at + s * 16), o = *reinterpret_cast<const v4f*>(co + at + s * 16),
                b = *reinterpret_cast<const v4f*>(cb + at + s * 16), cd = *reinterpret_cast<const v4f*>(cf + at + s * 16);
      const int64_t i = i0 + at + s * 16;
      float sums[3][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) sums[0][k] = sums[1][k] = sums[2][k] = 0.f;
#pragma unroll
      for (int jj = 0; jj < SN; ++jj) {
        const int64_t t = j0 + (wn * SN + jj) * 16 + r;
        float v[4], u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float sv = acc[s][jj][k] * f[jj], z = fmaf(a[k], sv, fmaf(o[k], X[jj], b[k]));
          const float p = scale[jj] == 0.f ? 0.f : __builtin_amdgcn_exp2f((z - top[jj]) * H_LOG2E) * scale[jj];
          v[k] = target[jj] == s * 16 + k ? own[jj] : p;
          sums[0][k] += v[k];
          sums[1][k] = fmaf(v[k], fmaf(mid, X[jj], sv), sums[1][k]);
          sums[2][k] = fmaf(v[k], X[jj], sums[2][k]);
          u[k] = target[jj] == s * 16 + k && A.own_target ? 0.f : A.raw_d ? v[k] : v[k] * cd[k] * gd[jj];
        }
        if (A.rowpart) rows[jj] += fmaf(v[0], o[0], v[1] * o[1]) + fmaf(v[2], o[2], v[3] * o[3]);
        if (A.d && t < A.t && i < A.mp) put_dz(A, t, i, u);
      }
      if (A.colpart)
#pragma unroll
        for (int c = 0; c < 3; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float w = sum16(sums[c][k]);
            if (r == 0) red[(wn * 3 + c) * BM + at + s * 16 + k] = w;
          }
    }
    float* rred = red + WN * 3 * BM;
    if (A.rowpart)
#pragma unroll
      for (int jj = 0; jj < SN; ++jj) {
        float w = rows[jj];
        w += shfl_xor_f(w, 16);
        w += shfl_xor_f(w, 32);
        if (kb == 0) rred[wm * BN + (wn * SN + jj) * 16 + r] = w;
      }
    __syncthreads();
    if (A.colpart)
      for (int k = threadIdx.x; k < 3 * BM; k += 64 * WM * WN) {
        const int c = k / BM, q = k - c * BM;
        if (i0 + q >= A.m) continue;
        float w = 0.f;
#pragma unroll
        for (int n = 0; n < WN; ++n) w += red[(n * 3 + c) * BM + q];
        A.colpart[(j0 / BN * 3 + c) * A.m + i0 + q] = w;
      }
    if (A.rowpart)
      for (int k = threadIdx.x; k < BN; k += 64 * WM * WN) {
        if (j0 + k >= A.t) continue;
        float w = 0.f;
#pragma unroll
        for (int n = 0; n < WM; ++n) w += rred[n * BN + k];
        A.rowpart[(j0 + k) * ((A.m + BM - 1) / BM) + i0 / BM] = w;
      }
  }
}

// dx's sum over the pieces: out[split][t][j] (+)= D[t][j] 2^-shift(rowmax[t]), the head's
// planes with their rows as depth.  A split has a sum of its own, so that the largest
// tile fills the CUs and nothing is joined before the end.  2048 tokens, 32768 rows of 4096
// columns: 420 us, 1.31 PFLOP/s, the matrix cores busy 57 %.  (With transposed planes in
// memory whole calls of 128256 rows, with gradients, took 6.12 ms, so 5.54.)
template <typename T, int BM, int BN, int WM, int WN, int AMODE>
__global__ __launch_bounds__(64 * WM * WN, 2) void head_dx_gemm_kernel(QGemm g, const uint32_t* __restrict__ rowmax,
                                                                       float* __restrict__ out, int64_t ldo, int splits,
                                                                       bool first) {
  constexpr int SM = BM / WM / 16, SN = BN / WN / 16;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[gemm_stages(BM, BN)][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, kb = lane >> 4;
  int split;
  int64_t i0, j0;
  v4f acc[SM][SN];
  q_gemm_tile<T, BM, BN, WM, WN, AMODE>(g, splits, lds, acc, split, i0, j0);
#pragma unroll
  for (int jj = 0; jj < SN; ++jj) {
    const int64_t t = j0 + (wn * SN + jj) * 16 + r;
    if (t >= g.N) continue;
    const float f = rowmax ? pow2(-pow2_shift(rowmax[t])) : 1.f;
    float* row = out + ((int64_t)split * g.N + t) * ldo;
    v4f old[SM];
#pragma unroll
    for (int s = 0; s < SM; ++s) {
      const int64_t i = i0 + (wm * SM + s) * 16 + 4 * kb;
      old[s] = (v4f){0.f, 0.f, 0.f, 0.f};
      if (!first && i < ldo) old[s] = *reinterpret_cast<const v4f*>(row + i);
    }
#pragma unroll
    for (int s = 0; s < SM; ++s) {
      const int64_t i = i0 + (wm * SM + s) * 16 + 4 * kb;
      if (i < ldo) *reinterpret_cast<v4f*>(row + i) = old[s] + acc[s][jj] * f;
    }
  }
}

struct DxPlan {
  int tile;   // 0: 256 x 256, 1: 256 x 128, 2: 128 x 128
  int64_t tiles;
  int splits;
};
// The tile and the splits of `steps` of the least time, by what a round of workgroups takes
// (24 us to begin and end, and a step 0.82, 0.55 and 0.62, the last with two on each CU: 512
// steps of 256 x 256 420 us, 98 of them 108; 196 of 256 x 128 136, 143 98; 143 of 128 x 128
// 112), and what a split's sum does, read and written (4 TB/s).
DxPlan dx_plan(int64_t n, int64_t T, int64_t steps) {
  constexpr int bm[3] = {256, 256, 128}, bn[3] = {256, 128, 128}, slots[3] = {256, 256, 512};
  constexpr double step_us[3] = {0.82, 0.55, 0.62};
  DxPlan best = {0, 0, 1};
  double least = 1e30;
  for (int tile = 0; tile < 3; ++tile) {
    const int64_t tiles = (n + bm[tile] - 1) / bm[tile] * ((T + bn[tile] - 1) / bn[tile]);
    for (int splits = 1; splits <= 32 && (splits == 1 || steps / splits >= 8); ++splits) {
      const double rounds = (double)((tiles * splits + slots[tile] - 1) / slots[tile]);
      const double us = rounds * (24.0 + (double)((steps + splits - 1) / splits) * step_us[tile]) + splits * (double)(T * n) * 8.0 / 4e6;
      if (us < least) {
        least = us;
        best = {tile, tiles, splits};
      }
    }
  }
  return best;
}

template <typename T, int AMODE>
hipError_t launch_dx(const QGemm& g, const uint32_t* rowmax, float* out, int64_t ldo, const DxPlan& p, bool first, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.splits));
  if (p.tile == 0)
    hipLaunchKernelGGL((head_dx_gemm_kernel<T, 256, 256, 2, 4, AMODE>), grid, dim3(512), 0, st, g, rowmax, out, ldo, p.splits, first);
  else if (p.tile == 1)
    hipLaunchKernelGGL((head_dx_gemm_kernel<T, 256, 128, 4, 2, AMODE>), grid, dim3(512), 0, st, g, rowmax, out, ldo, p.splits, first);
  else
    hipLaunchKernelGGL((head_dx_gemm_kernel<T, 128, 128, 2, 2, AMODE>), grid, dim3(256), 0, st, g, rowmax, out, ldo, p.splits, first);
  return hipGetLastError();
}

template <typename T, int AMODE, bool GRADS>
hipError_t launch(const QGemm& g, const PieceArgs& A, const uint32_t* rowmax, hipStream_t st) {
  const HeadTile tile = head_tile(g.M, g.N);
  const unsigned tiles = (unsigned)(((g.M + tile.rows - 1) / tile.rows) * ((g.N + tile.tokens - 1) / tile.tokens));
  if (tile.tokens == 256)
    hipLaunchKernelGGL((head_gemm_kernel<T, 256, 256, 2, 4, GRADS, AMODE>), dim3(tiles), dim3(512), 0, st, g, A, rowmax);
  else
    hipLaunchKernelGGL((head_gemm_kernel<T, 256, 128, 4, 2, GRADS, AMODE>), dim3(tiles), dim3(512), 0, st, g, A, rowmax);
  return hipGetLastError();
}
template <typename T, int AMODE>
hipError_t pick(const QGemm& g, const PieceArgs& A, const uint32_t* rowmax, bool grads, hipStream_t st) {
  return grads ? launch<T, AMODE, true>(g, A, rowmax, st) : launch<T, AMODE, false>(g, A, rowmax, st);
}

}  // namespace

// As the product's own rule: 256 x 256 where that gives three CUs in four a workgroup.
HeadTile head_tile(int64_t m, int64_t t) { return {256, (m + 255) / 256 * ((t + 255) / 256) >= 192 ? 256 : 128}; }

int head_dx_splits(int64_t n, int64_t t, int64_t rows, int npairs) { return dx_plan(n, t, rows / BK * npairs).splits; }
hipError_t launch_head_dx(const QGemm& g, const uint32_t* rowmax, float* out, int64_t ldo, int64_t rows, bool first,
                          hipStream_t st) {
  if (g.K % BK != 0 || g.K <= 0 || g.arows <= 0) return hipErrorInvalidValue;
  const DxPlan p = dx_plan(g.M, g.N, rows / BK * g.npairs);
  if (!g.lda) return launch_dx<OpF16, A_T_BLOCKS>(g, rowmax, out, ldo, p, first, st);
  return g.bf16 ? launch_dx<OpBf16, A_T_ROWS>(g, rowmax, out, ldo, p, first, st)
                : launch_dx<OpF16, A_T_ROWS>(g, rowmax, out, ldo, p, first, st);
}

hipError_t launch_head_gemm(const QGemm& g, const PieceArgs& A, const uint32_t* rowmax, bool grads, hipStream_t st) {
  if (g.K % BK != 0 || g.K <= 0) return hipErrorInvalidValue;
  if (!g.lda) return pick<OpF16, A_BLOCKS>(g, A, rowmax, grads, st);
  return g.bf16 ? pick<OpBf16, A_ROWS>(g, A, rowmax, grads, st) : pick<OpF16, A_ROWS>(g, A, rowmax, grads, st);
}

}  // namespace mpq
