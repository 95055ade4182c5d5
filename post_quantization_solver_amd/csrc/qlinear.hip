// A solved layer's product and its gradients: packing, operand preparation and
// the order of the launches (qlayer.h; products in qskinny.hip and qgemm.hip).
//
// Many rows: the layer's entries e (one affine per row; exact in 16 bits) or
// its weights a e + o (column groups) become 16-bit planes in the workspace, a
// block of rows at a time that stays in the last-level cache, and the product
// runs on the matrix cores; the affine, bias, activation and residual are its
// epilogue.
//
// Gradients (codes fixed): du = dy act'(pre);
//   dx = du W: one affine per row: (du a) e + du o', the second a number per
//        row of dx; groups: du times the weights' planes;
//   dW = du^T x, contracted as it leaves the product: d scale = sum_j e_ij dW_ij,
//        d offset = sum_j dW_ij over the columns of a group;
//   d bias = sum_t du.
//
// Roundings.  What is not exact in 16 bits (float32 x, du under an activation
// or times a scale, the weights of column groups) enters as float16 terms of
// itself times a power of two per row of the operand (qlayer.h): one term, 11
// bits, where a bfloat16 result is rounded to 8 anyway; two, 22 bits, for
// float16 and float32 results and for the float32 sums of the layer's gradients.
#include <string.h>
#include <algorithm>
#include <vector>
#include "qlayer.h"

namespace mpq {

namespace {

constexpr size_t QALIGN = 256;
inline size_t up(size_t x) { return (x + QALIGN - 1) / QALIGN * QALIGN; }
inline int64_t up64(int64_t x) { return (x + 63) / 64 * 64; }

// Rows of the layer unpacked at a time: their planes should stay in the 256 MB
// last-level cache between the two kernels.
constexpr int64_t Q_BLOCK_BYTES = (int64_t)128 << 20;

// ------------------------------------------------------------------ packing

__global__ __launch_bounds__(256) void q_pack_kernel(const int32_t* __restrict__ codes, QLayer L,
                                                     uint4* __restrict__ packed) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t total = (int64_t)L.tiles * L.chunks * 64;
  if (at >= total) return;
  const int lane = (int)(at & 63);
  const int64_t tc = at >> 6;
  const int64_t c = tc % L.chunks, i = tc / L.chunks * 16 + (lane & 15);
  const int steps = q_steps(L.fmt), kb = lane >> 4;
  const int64_t blk0 = c * steps * 4 + kb;   // step s: block blk0 + 4 s
  uint32_t w[4] = {0, 0, 0, 0};
  if (i < L.m) {
    if (L.fmt == QF_NIB || L.fmt == QF_BYTE) {
      const int bits = L.fmt == QF_NIB ? 4 : 8, count = steps * 8;
      for (int q = 0; q < count; ++q) {
        const int64_t j = (blk0 + q / 8 * 4) * 8 + q % 8;
        const int code = j < L.n ? safe_code(codes[i * L.n + j], L.K) : 0;
        // place of the q-th code (see qlayer.h)
        const int at = bits == 4 ? q / 8 * 8 + (q % 8 >> 1) + 4 * (q & 1) : q / 4 * 4 + (q % 4 >> 1) + 2 * (q & 1);
        const uint32_t v = (uint32_t)code << (at * bits & 31);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at * bits >> 5 == k) w[k] |= v;
      }
    } else {
      const int64_t B = L.n / 8;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t code = blk0 + 4 * s < B ? (uint32_t)safe_code(codes[i * B + blk0 + 4 * s], L.K) : 0u;
        if (L.fmt == QF_E8) code = L.map[code];
        w[s >> 1] |= code << (16 * (s & 1));
      }
    }
  }
  packed[at] = make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ operands

// The largest magnitude among a row's weights, bounded: max |a| max |e'| + |o'|
// over its groups; one wave per row.
__device__ __forceinline__ float row_bound(const QLayer& L, int64_t i, int lane) {
  float top = 0.f;
  const float mid = q_centre(L);
  for (int k = lane; k < L.K; k += 64) top = fmaxf(top, fabsf(L.levels[k] - mid));   // groups have d = 1
  for (int o = 32; o; o >>= 1) top = fmaxf(top, shfl_xor_f(top, o));
  float w = 0.f;
  bool odd = false;
  for (int64_t g = lane; g < L.G; g += 64) {
    const float a = L.scale[i * L.G + g], o = fmaf(a, mid, L.offset ? L.offset[i * L.G + g] : 0.f);
    const float b = fabsf(a) * top + fabsf(o);
    odd |= !(b <= 3.4028235e38f);
    w = fmaxf(w, b);
  }
  for (int o = 32; o; o >>= 1) w = fmaxf(w, shfl_xor_f(w, o));
  return __ballot(odd) ? 0.f : w;   // a row that is not finite keeps factor 1
}

__device__ __forceinline__ void weight_terms(const float* v, v4u* out) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t a[2], b[2];
    f16_terms(v[2 * q], a);
    f16_terms(v[2 * q + 1], b);
    out[0][q] = pack2(a[0], b[0]);
    out[1][q] = pack2(a[1], b[1]);
  }
}

struct PrepArgs {
  const void* x; int64_t ldx;
  int dtype;
  int64_t t, rows;      // rows t .. rows - 1 of the planes are zeros
  int64_t n, Kp;        // columns n .. Kp - 1 too
  uint16_t* out; int64_t plane;
  int planes;           // 0: none
  bool raw;             // 16-bit x as it is; else float16 terms of x times 2^pow2_shift(rowmax)
  bool frags;           // planes in the order of qskinny.hip's operands, else of qgemm.hip's
  bool vec;             // rows of x can be read 8 elements at a time
  int segs;             // workgroups per row (1 where a row's sum or maximum is wanted)
  uint32_t* rowmax;
  float* sum;
  QLayer L; uint32_t* refs;
};

// Workgroups 0 .. rows segs - 1: a row (or a part) of x, its planes, and
// optionally its sum.  The ones after them, a wave per row of the layer: refs =
// its weights' bound.
__global__ __launch_bounds__(256) void q_prep_kernel(PrepArgs A) {
  __shared__ float red[2][4];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t row = blockIdx.x / A.segs;
  if (row >= A.rows) {
    const int64_t i = (blockIdx.x - A.rows * A.segs) * 4 + wave;
    if (i >= A.L.m) return;
    const float b = row_bound(A.L, i, lane);
    if (lane == 0) A.refs[i] = __float_as_uint(b);
    return;
  }
  const int seg = (int)(blockIdx.x - row * A.segs);
  const bool live = row < A.t;
  auto load8 = [&](int64_t j, float* v) {
    const int have = live ? (int)max((int64_t)0, min((int64_t)8, A.n - j)) : 0;
    load4(A.x, row * A.ldx + j, A.dtype, A.vec, min(have, 4), v);
    load4(A.x, row * A.ldx + j + 4, A.dtype, A.vec, max(have - 4, 0), v + 4);
  };
  uint32_t top = 0;
  if (A.sum || (A.planes && !A.raw)) {
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
    for (int w = 0; w < 4; ++w) top = max(top, __float_as_uint(red[1][w]));
    if (threadIdx.x == 0 && live) {
      if (A.sum) A.sum[row] = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
      if (A.planes && !A.raw) A.rowmax[row] = top;
    }
  }
  if (!A.planes) return;
  const float f = pow2(pow2_shift(top));
  for (int64_t j = ((int64_t)seg * 256 + threadIdx.x) * 8; j < A.Kp; j += (int64_t)A.segs * 256 * 8) {
    float v[8];
    load8(j, v);
    v4u o[2];
    if (A.raw) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[0][q] = A.dtype == DT_BF16 ? OpBf16::pack(v[2 * q], v[2 * q + 1]) : OpF16::pack(v[2 * q], v[2 * q + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
      weight_terms(v, o);
    }
    // operand order: step of 32 columns by step, lane (j / 8 % 4) 16 + row % 16
    uint16_t* dst = A.out + (A.frags ? ((row >> 4) * (A.Kp >> 5) + (j >> 5)) * 512 + ((j >> 3 & 3) * 16 + (row & 15)) * 8
                                     : q_at(row, j, A.Kp));
    *reinterpret_cast<v4u*>(dst) = o[0];
    if (A.planes > 1) *reinterpret_cast<v4u*>(dst + A.plane) = o[1];
  }
}

// Eight weights of row i from their entries, times f.
__device__ __forceinline__ void weights8(const QLayer& L, int64_t i, int64_t j0, v4u e, float mid, float f, float* v) {
  if (L.group % 8 == 0 || L.G == 1) {   // one group
    const int64_t g = i * L.G + (L.G > 1 ? min(j0, L.n - 1) / L.group : 0);
    const float a = L.scale[g], o = fmaf(a, mid, L.offset ? L.offset[g] : 0.f);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = j0 + q < L.n ? fmaf(a, OpF16::val(q & 1 ? e[q >> 1] >> 16 : e[q >> 1] & 0xffffu), o) * f : 0.f;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t g = i * L.G + min(j0 + q, L.n - 1) / L.group;
      const float a = L.scale[g], o = fmaf(a, mid, L.offset ? L.offset[g] : 0.f);
      v[q] = j0 + q < L.n ? fmaf(a, OpF16::val(q & 1 ? e[q >> 1] >> 16 : e[q >> 1] & 0xffffu), o) * f : 0.f;
    }
  }
}
// Rows tile0 * 16 .. of the layer as planes of Kp columns: entries (planes = 0),
// or float16 terms of the weights times 2^pow2_shift(refs).  A wave per chunk of
// a tile.
template <int FMT, typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void q_unpack_kernel(QLayer L, int tile0, int tiles, int64_t Kp, int planes,
                                                              const uint32_t* __restrict__ refs,
                                                              uint16_t* __restrict__ out, int64_t plane) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int lane = threadIdx.x & 63, wave = wave_id();
  q_lut_fill<FMT, T>(L, lds, 64 * WAVES);
  if (FMT == QF_E8) q_lut_wait<0>();
  __syncthreads();
  const float mid = q_centre(L);
  const int64_t total = (int64_t)tiles * L.chunks;
  for (int64_t w = (int64_t)blockIdx.x * WAVES + wave; w < total; w += (int64_t)gridDim.x * WAVES) {
    const int tl = (int)(w / L.chunks), c = (int)(w - (int64_t)tl * L.chunks);
    const uint4 code = L.packed[((size_t)(tile0 + tl) * L.chunks + c) * 64 + lane];
    const int64_t row = tl * 16 + (lane & 15), i = (int64_t)tile0 * 16 + row;
    const float f = planes ? pow2(pow2_shift(refs[min(i, L.m - 1)])) : 1.f;
#pragma unroll
    for (int s = 0; s < q_steps(FMT); ++s) {
      const int64_t j0 = (((int64_t)c * q_steps(FMT) + s) * 4 + (lane >> 4)) * 8;
      v4u e = q_decode<FMT, T>(L, lds, code, s);
      if (j0 >= Kp) continue;
      uint16_t* dst = out + q_at(row, j0, Kp);
      if (planes == 0) {
        // columns past the last hold zero, whatever their codes
        if (j0 + 8 > L.n) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (j0 + q >= L.n) e[q >> 1] &= q & 1 ? 0xffffu : 0xffff0000u;
        }
        *reinterpret_cast<v4u*>(dst) = e;
      } else if constexpr (T::HALF) {
        float v[8];
        v4u o[2];
        weights8(L, min(i, L.m - 1), j0, e, mid, f, v);
        weight_terms(v, o);
        *reinterpret_cast<v4u*>(dst) = o[0];
        if (planes > 1) *reinterpret_cast<v4u*>(dst + plane) = o[1];
      }
    }
  }
}

// The transpose, float16: plane rows are the layer's columns, mp (m padded
// with zeros to 64) entries or weights each.  A workgroup unpacks 16 WAVES rows
// of one chunk, 32 columns at a time, through LDS; a lane's eight columns are
// spread over LDS rows padded by 16 bytes, so that the sixteen rows of a store
// share no bank with the next column's.
template <int FMT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void q_unpack_t_kernel(QLayer L, int64_t mp, int planes,
                                                                const uint32_t* __restrict__ refs,
                                                                uint16_t* __restrict__ out, int64_t plane,
                                                                int lut_words) {
  using T = OpF16;
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int ROWS = 16 * WAVES, PITCH = ROWS + 8;
  uint16_t* tl = reinterpret_cast<uint16_t*>(lds + lut_words);   // 32 columns x PITCH
  const int lane = threadIdx.x & 63, wave = wave_id();
  q_lut_fill<FMT, T>(L, lds, 64 * WAVES);
  if (FMT == QF_E8) q_lut_wait<0>();
  __syncthreads();
  const float mid = q_centre(L);
  const int64_t strips = (mp + ROWS - 1) / ROWS, total = strips * L.chunks;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t strip = w / L.chunks;
    const int c = (int)(w - strip * L.chunks);
    const int64_t tile = strip * WAVES + wave;
    const bool live = tile < L.tiles;
    uint4 code = make_uint4(0, 0, 0, 0);
    if (live) code = L.packed[((size_t)tile * L.chunks + c) * 64 + lane];
    const int64_t i = tile * 16 + (lane & 15), is = min(i, L.m - 1);
    const float f = planes ? pow2(pow2_shift(refs[is])) : 1.f;
#pragma unroll 1
    for (int s = 0; s < q_steps(FMT); ++s) {
      // (the step is not unrolled: its word is picked, so that one copy of the decoder remains)
      const uint32_t ws[4] = {code.x, code.y, code.z, code.w};
      uint4 cs = code;
      if (FMT == QF_NIB) {
        cs.x = s == 0 ? ws[0] : s == 1 ? ws[1] : s == 2 ? ws[2] : ws[3];
      } else if (FMT == QF_BYTE) {
        cs.x = s == 0 ? ws[0] : ws[2];
        cs.y = s == 0 ? ws[1] : ws[3];
      } else {
        const uint32_t x = s < 2 ? ws[0] : s < 4 ? ws[1] : s < 6 ? ws[2] : ws[3];
        cs.x = s & 1 ? x >> 16 : x;
      }
      v4u o[2];
      o[0] = q_decode<FMT, T>(L, lds, cs, 0);
      if (planes > 0) {
        float v[8];
        weights8(L, is, (((int64_t)c * q_steps(FMT) + s) * 4 + (lane >> 4)) * 8, o[0], mid, f, v);
        weight_terms(v, o);
      }
      if (i >= L.m) o[0] = o[1] = (v4u){0u, 0u, 0u, 0u};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p > 0 && p >= planes) break;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          tl[((lane >> 4) * 8 + q) * PITCH + wave * 16 + (lane & 15)] =
              (uint16_t)(q & 1 ? o[p][q >> 1] >> 16 : o[p][q >> 1] & 0xffffu);
        __syncthreads();
        constexpr int PIECES = ROWS / 8;
        for (int k = threadIdx.x; k < 32 * PIECES; k += 64 * WAVES) {
          const int col = k / PIECES, piece = k - col * PIECES;
          const int64_t j = ((int64_t)c * q_steps(FMT) + s) * 32 + col;
          const int64_t r = strip * ROWS + piece * 8;
          if (j < L.n && r < mp)
            *reinterpret_cast<v4u*>(out + p * plane + q_at(j, r, mp)) =
                *reinterpret_cast<const v4u*>(tl + col * PITCH + piece * 8);
        }
        __syncthreads();
      }
    }
  }
}

// ------------------------------------------------------------------ gradients

// Tiles of 64 x 64: thread (tid / 16, tid % 16) has rows tid / 16 + 16 k, four
// consecutive columns.
struct DuArgs {
  const void* dy; int64_t lddy;
  const void* pre; int64_t ldpre;
  const void* x; int64_t ldx;
  int act, dtype;
  bool vec_du, vec_x;                 // 4-element alignment of dy and pre, of x
  int64_t t, m, n;
  QLayer L;
  bool want_d, want_t;
  // largest magnitudes (bits): du times the layer row's factor per token, du
  // per layer row, x per column; refs: the layer rows' bounds (groups)
  uint32_t *dmax, *tmax, *xmax, *refs;
  // du times the factor, float16 terms, t rows of mp
  uint16_t* d; int64_t plane_d, mp; int planes_d;
  float* rowpart; int64_t rowtiles;   // t x rowtiles: sums of du o' over 64 columns (nullptr: none)
  // du^T, float16 terms, m rows of tp
  uint16_t* dt; int64_t plane_t, tp; int planes_t;
  float* biaspart;                    // (tp / 64) x m: sums of du over 64 rows
  // x^T, float16 terms, n rows of tp
  uint16_t* xt; int64_t plane_x; int planes_x;
  int64_t du_blocks, xtiles;          // 64 x 64 tiles of du, column tiles of x
};

// What the rows of du are multiplied by for dx: the scale itself (one affine
// per row), or the inverse of what the weights' planes are scaled by.
__device__ __forceinline__ float du_factor(const DuArgs& A, int64_t i) {
  return A.L.G == 1 ? A.L.scale[i] : pow2(-pow2_shift(A.refs[i]));
}

// Four values of du at row t, columns i ..
__device__ __forceinline__ void load_du(const DuArgs& A, int64_t t, int64_t i, float* v) {
  const int live = t < A.t ? (int)max((int64_t)0, min((int64_t)4, A.m - i)) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = 0.f;
  if (live == 0) return;
  load4(A.dy, t * A.lddy + i, A.dtype, A.vec_du, live, v);
  if (A.act != ACT_NONE) {
    float u[4];
    load4(A.pre, t * A.ldpre + i, A.dtype, A.vec_du, live, u);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < live) v[k] *= act_slope(A.act, u[k]);
  }
}
__device__ __forceinline__ void load_x(const DuArgs& A, int64_t t, int64_t j, float* v) {
  const int live = t < A.t ? (int)max((int64_t)0, min((int64_t)4, A.n - j)) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = 0.f;
  if (live) load4(A.x, t * A.ldx + j, A.dtype, A.vec_x, live, v);
}

// Clears the maxima and fills refs (groups; a wave per row).
__global__ __launch_bounds__(256) void q_grad_init_kernel(DuArgs A) {
  const int lane = threadIdx.x & 63;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < max(max(A.t, A.m), A.n); k += (int64_t)gridDim.x * 256) {
    if (k < A.t) A.dmax[k] = 0;
    if (k < A.m) A.tmax[k] = 0;
    if (k < A.n) A.xmax[k] = 0;
  }
  if (A.L.G > 1)
    for (int64_t i = (int64_t)blockIdx.x * 4 + wave_id(); i < A.m; i += (int64_t)gridDim.x * 4) {
      const float b = row_bound(A.L, i, lane);
      if (lane == 0) A.refs[i] = __float_as_uint(b);
    }
}

// The maxima (integer maxima of magnitudes' bits: in any order the same).
__global__ __launch_bounds__(256) void q_grad_scan_kernel(DuArgs A) {
  __shared__ uint32_t cm[4][64];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4, wave = wave_id();
  const bool is_x = blockIdx.x >= A.du_blocks;
  const int64_t b = is_x ? blockIdx.x - A.du_blocks : blockIdx.x, ct = is_x ? A.xtiles : A.rowtiles;
  const int64_t t0 = b / ct * 64, i = (b % ct) * 64 + cx * 4;
  uint32_t col[4] = {0, 0, 0, 0};
  float f[4] = {1.f, 1.f, 1.f, 1.f};
  const bool rows = !is_x && A.want_d;
  if (rows)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < A.m) f[k] = du_factor(A, i + k);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t t = t0 + ry + 16 * k;
    float v[4];
    if (is_x) load_x(A, t, i, v); else load_du(A, t, i, v);
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      col[q] = max(col[q], abs_bits(v[q]));
      top = max(top, abs_bits(v[q] * f[q]));
    }
    if (rows) {
      top = max(top, (uint32_t)dpp_i<DPP_XOR1>((int)top));
      top = max(top, (uint32_t)dpp_i<DPP_XOR2>((int)top));
      top = max(top, (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)top));
      top = max(top, (uint32_t)dpp_i<DPP_MIRROR>((int)top));
      if (cx == 0 && t < A.t) atomicMax(A.dmax + t, top);
    }
  }
  if (!is_x && !A.want_t) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    col[q] = max(col[q], (uint32_t)shfl_xor_i((int)col[q], 16));
    col[q] = max(col[q], (uint32_t)shfl_xor_i((int)col[q], 32));
    if ((threadIdx.x & 63) < 16) cm[wave][cx * 4 + q] = col[q];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t j = (b % ct) * 64 + threadIdx.x;
    const uint32_t top = max(max(cm[0][threadIdx.x], cm[1][threadIdx.x]), max(cm[2][threadIdx.x], cm[3][threadIdx.x]));
    if (j < (is_x ? A.n : A.m)) atomicMax((is_x ? A.xmax : A.tmax) + j, top);
  }
}

// Four float16 terms of v at p[0 .. 3].
__device__ __forceinline__ void put_terms(uint16_t* p, int64_t plane, int planes, const float* v) {
  uint32_t b[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) f16_terms(v[k], b[k]);
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(b[0][0], b[1][0]), pack2(b[2][0], b[3][0]));
  if (planes > 1)
    *reinterpret_cast<uint2*>(p + plane) = make_uint2(pack2(b[0][1], b[1][1]), pack2(b[2][1], b[3][1]));
}
__device__ __forceinline__ float sum16(float s) {
  s += dpp_f<DPP_XOR1>(s);
  s += dpp_f<DPP_XOR2>(s);
  s += dpp_f<DPP_HALF_MIRROR>(s);
  s += dpp_f<DPP_MIRROR>(s);
  return s;
}

// A 64 x 64 tile of du (its planes, its transpose's, its row and column sums)
// or of x (its transpose's planes).
__global__ __launch_bounds__(256) void q_grad_tile_kernel(DuArgs A) {
  __shared__ float tl[64][65];
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const bool is_x = blockIdx.x >= A.du_blocks;
  const int64_t b = is_x ? blockIdx.x - A.du_blocks : blockIdx.x, ct = is_x ? A.xtiles : A.rowtiles;
  const int64_t t0 = b / ct * 64, i0 = (b % ct) * 64, i = i0 + cx * 4;
  float f[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (!is_x && A.want_d)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < A.m) {
        f[k] = du_factor(A, i + k);
        if (A.rowpart) o[k] = fmaf(A.L.scale[i + k], q_centre(A.L), A.L.offset ? A.L.offset[i + k] : 0.f);
      }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t t = t0 + ry + 16 * k;
    float v[4];
    if (is_x) load_x(A, t, i, v); else load_du(A, t, i, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) tl[ry + 16 * k][cx * 4 + q] = v[q];
    if (is_x || !A.want_d) continue;
    if (A.rowpart) {
      const float s = sum16(fmaf(v[0], o[0], v[1] * o[1]) + fmaf(v[2], o[2], v[3] * o[3]));
      if (cx == 0 && t < A.t) A.rowpart[t * A.rowtiles + b % ct] = s;
    }
    if (t < A.t) {
      const float g = pow2(pow2_shift(A.dmax[t]));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] * f[q] * g;   // (as the scan took it: f g alone may overflow)
      put_terms(A.d + q_at(t, i, A.mp), A.plane_d, A.planes_d, v);
    }
  }
  if (!is_x && !A.want_t) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = i0 + ry + 16 * k;   // row of the transpose: sixteen lanes have its 64 tokens
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = tl[cx * 4 + q][ry + 16 * k];
    const float s = sum16((v[0] + v[1]) + (v[2] + v[3]));
    if (r >= (is_x ? A.n : A.m)) continue;
    if (!is_x && cx == 0) A.biaspart[t0 / 64 * A.m + r] = s;
    const float g = pow2(pow2_shift(is_x ? A.xmax[r] : A.tmax[r]));
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] *= g;
    if (is_x) put_terms(A.xt + q_at(r, t0 + cx * 4, A.tp), A.plane_x, A.planes_x, v);
    else put_terms(A.dt + q_at(r, t0 + cx * 4, A.tp), A.plane_t, A.planes_t, v);
  }
}

// d bias of row r, and du o' per token: added up in order in float64.
__device__ __forceinline__ void add_bias(const DuArgs& A, int64_t r, float* __restrict__ dbias) {
  if (r >= A.m) return;
  double s = 0.0;
  for (int64_t k = 0; k < A.tp / 64; ++k) s += (double)A.biaspart[k * A.m + r];
  dbias[r] = (float)s;
}
__global__ __launch_bounds__(256) void q_grad_rowsum_kernel(DuArgs A, float* __restrict__ rowadd) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= A.t) return;
  double s = 0.0;
  for (int64_t k = 0; k < A.rowtiles; ++k) s += (double)A.rowpart[t * A.rowtiles + k];
  rowadd[t] = (float)s;
}

// The contraction's parts, added up in order in float64: sixteen lanes per (row, group).
__global__ __launch_bounds__(256) void q_contract_finish_kernel(QLayer L, const float2* __restrict__ part, int splits,
                                                                int64_t rows, int64_t blocks, int64_t row0,
                                                                float* __restrict__ dscale,
                                                                float* __restrict__ doffset, DuArgs A,
                                                                float* __restrict__ dbias) {
  const int64_t own = (rows * L.G + 15) / 16;
  if (blockIdx.x >= own) {   // d bias
    add_bias(A, (blockIdx.x - own) * 256 + threadIdx.x, dbias);
    return;
  }
  const int lane = threadIdx.x & 15;
  const int64_t w = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (w >= rows * L.G) return;
  const int64_t row = w / L.G, g = w - row * L.G;
  const int64_t b0 = g * (L.group / Q_CONTRACT), b1 = L.G == 1 ? blocks : min(blocks, b0 + L.group / Q_CONTRACT);
  double se = 0.0, s1 = 0.0;
  for (int s = 0; s < splits; ++s)
    for (int64_t b = b0 + lane; b < b1; b += 16) {
      const float2 p = part[((size_t)s * rows + row) * blocks + b];
      se += (double)p.x;
      s1 += (double)p.y;
    }
  for (int o = 8; o; o >>= 1) {
    se += shfl_d(se, (int)(threadIdx.x & 63) ^ o);
    s1 += shfl_d(s1, (int)(threadIdx.x & 63) ^ o);
  }
  if (lane == 0) {
    dscale[(row0 + row) * L.G + g] = (float)se;
    doffset[(row0 + row) * L.G + g] = (float)s1;
  }
}

// Groups that are no multiple of 64 columns: the contraction of a dW in memory.
// d scale and d offset of `rows` rows from row0 on: a wave per (row, group).
__global__ __launch_bounds__(256) void q_affine_grad_kernel(QLayer L, const float* __restrict__ dW, int64_t ldw,
                                                            int64_t row0, int64_t rows, float* __restrict__ dscale,
                                                            float* __restrict__ doffset, DuArgs A,
                                                            float* __restrict__ dbias) {
  const int64_t own = (rows * L.G + 3) / 4;
  if (blockIdx.x >= own) {   // d bias
    add_bias(A, (blockIdx.x - own) * 256 + threadIdx.x, dbias);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= rows * L.G) return;
  const int64_t row = w / L.G, g = w - row * L.G, i = row0 + row;
  const int64_t j0 = g * L.group, j1 = min(L.n, j0 + L.group);
  double se = 0.0, s1 = 0.0;
  for (int64_t q = j0 / 4 + lane; q * 4 < j1; q += 64) {
    float e[4];
    q_entries4(L, q_code4(L, i, q * 4), q * 4, e);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t j = q * 4 + k;
      if (j < j0 || j >= j1) continue;
      const float d = dW[row * ldw + j];
      se += (double)(e[k] * d);
      s1 += (double)d;
    }
  }
  for (int o = 32; o; o >>= 1) {
    se += shfl_d(se, lane ^ o);
    s1 += shfl_d(s1, lane ^ o);
  }
  if (lane == 0) {
    dscale[i * L.G + g] = (float)se;
    doffset[i * L.G + g] = (float)s1;
  }
}

// ------------------------------------------------------------------ launches

template <typename T>
hipError_t unpack(const QLayer& L, int tile0, int tiles, int64_t Kp, int planes, const uint32_t* refs, uint16_t* out,
                  int64_t plane, hipStream_t st) {
  const size_t shared = (size_t)q_lut_words(L.fmt, (L.lut_entries + 3) / 4 * 4) * 4;
  const int64_t waves = (int64_t)tiles * L.chunks;
  auto grid = [&](int per, int most) { return dim3((unsigned)std::min<int64_t>((waves + per - 1) / per, most)); };
  switch (L.fmt) {
    case QF_NIB:
      hipLaunchKernelGGL((q_unpack_kernel<QF_NIB, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, refs, out, plane);
      break;
    case QF_BYTE:
      hipLaunchKernelGGL((q_unpack_kernel<QF_BYTE, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, refs, out, plane);
      break;
    case QF_E8:   // the table fills a CU's LDS: one workgroup of 16 waves each
      hipLaunchKernelGGL((q_unpack_kernel<QF_E8, T, 16>), grid(16, 256), dim3(1024), shared, st, L, tile0, tiles, Kp,
                         planes, refs, out, plane);
      break;
    default:
      hipLaunchKernelGGL((q_unpack_kernel<QF_VEC, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, refs, out, plane);
  }
  return hipGetLastError();
}

hipError_t unpack_t(const QLayer& L, int64_t mp, int planes, const uint32_t* refs, uint16_t* out, int64_t plane,
                    hipStream_t st) {
  const int lut = q_lut_words(L.fmt, (L.lut_entries + 3) / 4 * 4);
  auto go = [&](auto kernel, int waves, int most) {
    const int64_t total = (mp + 16 * waves - 1) / (16 * waves) * L.chunks;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(total, most)), dim3(64 * waves),
                       (size_t)lut * 4 + (size_t)32 * (16 * waves + 8) * 2, st, L, mp, planes, refs, out, plane, lut);
  };
  switch (L.fmt) {
    case QF_NIB: go(q_unpack_t_kernel<QF_NIB, 4>, 4, 2048); break;
    case QF_BYTE: go(q_unpack_t_kernel<QF_BYTE, 4>, 4, 2048); break;
    case QF_E8: go(q_unpack_t_kernel<QF_E8, 8>, 8, 256); break;
    default: go(q_unpack_t_kernel<QF_VEC, 4>, 4, 2048); break;
  }
  return hipGetLastError();
}

// Token counts up to which the product reads the packed codes (one affine per
// row, or groups of whole chunks; other groups always unpack).  Beyond, every 64
// tokens decode the layer once more, and laying the planes out once is cheaper.
// Measured, few-row product | planes and tiles, 4096 x 14336: E8 bfloat16 58 | 61
// us at 128 tokens, 84 | 77 at 192, float32 85 | 87 at 96, 109 | 90 at 128; four
// bits bfloat16 71 | 83 at 192, 93 | 85 at 256; 8 bits 81 | 97 at 192, 104 | 100 at
// 256, float32 79 | 105 at 96, 103 | 108 at 128; groups of 128, whose planes hold
// weights (two terms but for bfloat16): float16 156 | 213 at 384 (14336 x 4096
// 235 | 211 at 512), float32 188 | 251 at 192.  The planes take 18 us and more
// however small the layer: 1024 x 1024 at 384 tokens 17 | 20 (E8), 12 | 21 (four
// bits), 24 | 28 (float32), at 768 25 | 23, 17 | 24, 44 | 32; 8 bits at 768 20 | 26.
// A generic codebook's entries come from memory, and from 81 tokens on (float32:
// 65) a large layer of it would be better off with planes: 87 | 70 at 96, 93 | 71 at
// 128 (4096 x 4096 31 | 34, 33 | 34).  It takes E8's counts all the same: a
// workspace's size knows the codes, not the codebook, and planes take 128 MB.
constexpr int64_t Q_SMALL_TOKENS = 1024, Q_SMALL_WORK = 3ll << 27;

bool use_skinny(const QLinearArgs& A) {
  if (!q_skinny_ok(A.L)) return false;
  if (A.t <= Q_SMALL_TOKENS && A.t * A.L.m * A.L.n <= Q_SMALL_WORK) return true;
  const bool scalar = A.L.fmt == QF_NIB || A.L.fmt == QF_BYTE, grouped = A.L.G > 1;
  if (A.dtype == DT_F32) return A.t <= (grouped ? 192 : 96);
  return A.t <= (grouped && A.dtype == DT_F16 ? 384 : scalar ? 192 : 128);
}

// Elements of x up to which the few-row product reads it in place.
// Measured, in place | laid out first (E8): 4096 columns, 2 tokens 8.7 | 11.5 us,
// 16 tokens 10.7 | 11.8, 32 tokens 13.6 | 12.5; 8192 columns, 8 tokens 11.5 |
// 12.9, 13 tokens 12.6 | 13.0, 16 tokens 13.8 | 12.9; 14336 columns, 8 tokens 16.0
// | 16.3, 13 tokens 18.3 | 16.7.  8 bits: 4096 columns, 16 tokens 8.1 | 9.3, 32
// tokens 11.6 | 10.5; 8192 columns, 13 tokens 10.7 | 11.6, 16 tokens 11.9 | 11.7; 14336
// columns, 8 tokens 13.6 | 15.3, 13 tokens 15.7 | 15.4; four bits and generic alike.
constexpr int64_t Q_DIRECT = 7 << 14;

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

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

bool whole_quads(const void* p, int64_t ld, int dtype) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (dtype == DT_F32 ? 16 : 8) == 0 && ld % 4 == 0);
}

// Forward: lays out the workspace (which depends on the shapes and types
// alone) and, with a base, launches.
hipError_t forward(const QLinearArgs& A, char* base, size_t* bytes, hipStream_t st) {
  const QLayer& L = A.L;
  const bool skinny = use_skinny(A), grouped = L.G > 1, weights = grouped && !skinny;
  // the few-row product reads whole chunks
  const int64_t Kp = skinny ? (int64_t)L.chunks * q_chunk(L.fmt) : up64(L.n);
  // x: its own 16 bits, or float16 terms (float32; bfloat16 against weights)
  const int XP = A.dtype == DT_F32 ? 2 : 1;
  const bool raw = A.dtype == DT_F16 || (A.dtype == DT_BF16 && !weights);
  const bool aligned = reinterpret_cast<uintptr_t>(A.x) % 16 == 0 && A.ldx % 8 == 0 && A.ldx <= (1 << 20);
  // Few rows: see Q_DIRECT.  Many: the product's tiles read x in place as they do
  // operand order (2048 tokens, 4096 x 14336 E8 224 us, laid out first 235; 4096 x
  // 4096 four bits 79, 83).
  const bool direct = raw && aligned && (skinny ? L.n % 8 == 0 && A.t * L.n <= Q_DIRECT : L.n % 64 == 0);
  const bool bf16 = raw && A.dtype == DT_BF16;
  const int WP = !weights ? 0 : A.dtype == DT_BF16 ? 1 : 2;   // terms of a weight (0: entries)
  const bool sums = !skinny && !grouped && L.has_offset();
  Carve W{base};
  const int64_t xrows = up16(A.t), plane = xrows * Kp;
  uint16_t* xp = W.take<uint16_t>((size_t)XP * plane * 2);
  float* xs = W.take<float>((size_t)A.t * 4);
  uint32_t* rowmax = W.take<uint32_t>((size_t)A.t * 4);
  uint32_t* refs = W.take<uint32_t>((size_t)L.m * 4);
  const int per = WP ? WP : 1;
  int64_t rows = std::max<int64_t>(256, Q_BLOCK_BYTES / (per * Kp * 2) / 256 * 256);
  rows = std::min(rows, (int64_t)L.tiles * 16);
  QGemm g;
  memset(&g, 0, sizeof(g));
  q_pairs(g, per, XP);
  uint16_t* wp = nullptr;
  float* part = nullptr;
  if (!skinny) {
    wp = W.take<uint16_t>((size_t)per * rows * Kp * 2);
    size_t ps = 0;
    for (int64_t r0 = 0; r0 < L.m; r0 += rows)
      ps = std::max(ps, q_gemm_workspace(std::min(rows, L.m - r0), A.t, Kp, g.npairs));
    part = W.take<float>(ps);
  }
  if (bytes) *bytes = W.at;
  if (!base) return hipSuccess;

  hipError_t e;
  if (!direct || sums || weights) {
    PrepArgs P;
    memset(&P, 0, sizeof(P));
    P.x = A.x; P.ldx = A.ldx;
    P.dtype = A.dtype;
    P.t = A.t; P.rows = direct ? A.t : xrows;
    P.n = L.n; P.Kp = Kp;
    P.out = xp; P.plane = plane;
    P.planes = direct ? 0 : XP;
    P.raw = raw;
    P.frags = skinny;
    P.vec = reinterpret_cast<uintptr_t>(A.x) % 16 == 0 && A.ldx % 4 == 0;
    P.rowmax = rowmax;
    P.sum = sums ? xs : nullptr;
    P.L = L; P.refs = refs;
    P.segs = !raw || sums ? 1 : (int)std::max<int64_t>(1, std::min((Kp + 2047) / 2048, 512 / P.rows));
    const int64_t blocks = P.rows * P.segs + (weights ? (L.m + 3) / 4 : 0);
    hipLaunchKernelGGL(q_prep_kernel, dim3((unsigned)blocks), dim3(256), 0, st, P);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const uint16_t* x = direct ? static_cast<const uint16_t*>(A.x) : xp;
  QOut O;
  memset(&O, 0, sizeof(O));
  O.y = A.y; O.ldy = A.ldy;
  O.pre = A.pre; O.ldpre = A.ldpre;
  O.res = A.res; O.ldres = A.ldres;
  O.bias = A.bias;
  O.rowmax = raw ? nullptr : rowmax;
  O.act = A.act;
  O.dtype = A.dtype;
  O.mid = -1;
  O.rows = A.t;
  O.cols = L.m;
  O.vec = whole_quads(A.y, A.ldy, A.dtype) && whole_quads(A.pre, A.ldpre, A.dtype) &&
          whole_quads(A.res, A.ldres, A.dtype);
  if (skinny)
    return launch_q_skinny(L, x, direct ? A.ldx : 0, plane, A.t, XP, bf16, O, st);
  const int es = A.dtype == DT_F32 ? 4 : 2;
  for (int64_t r0 = 0; r0 < L.m; r0 += rows) {
    const int64_t nr = std::min(rows, L.m - r0);
    const int tiles = (int)((nr + 15) / 16);
    e = bf16 ? unpack<OpBf16>(L, (int)(r0 / 16), tiles, Kp, WP, refs, wp, rows * Kp, st)
             : unpack<OpF16>(L, (int)(r0 / 16), tiles, Kp, WP, refs, wp, rows * Kp, st);
    if (e != hipSuccess) return e;
    g.A = wp; g.planeA = rows * Kp;
    g.B = x; g.ldb = direct ? A.ldx : 0; g.planeB = plane;
    g.M = nr; g.N = A.t; g.K = Kp;
    g.bf16 = bf16;
    g.O = O;
    g.O.cols = nr;
    g.O.y = static_cast<char*>(A.y) + r0 * es;
    if (A.pre) g.O.pre = static_cast<char*>(A.pre) + r0 * es;
    if (A.res) g.O.res = static_cast<const char*>(A.res) + r0 * es;
    if (A.bias) g.O.bias = A.bias + r0;
    if (weights) {
      g.O.colmax = refs + r0;
    } else {
      g.O.colscale = L.scale + r0;
      g.O.coloff = L.offset ? L.offset + r0 : nullptr;
      g.O.rowadd = sums ? xs : nullptr;
      g.O.levels = L.levels;
      g.O.mid = L.fmt == QF_NIB || L.fmt == QF_BYTE ? L.K / 2 : -1;
    }
    // (the column blocks start at multiples of 256: their alignment is the whole's)
    if ((e = launch_q_gemm(g, part, st)) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t backward(const QLinearGrad& A, char* base, size_t* bytes, hipStream_t st) {
  const QLayer& L = A.L;
  const bool grouped = L.G > 1, contract = !grouped || L.group % Q_CONTRACT == 0;
  const int64_t mp = up64(L.m), tp = up64(A.t);
  const int XP = A.dtype == DT_F32 ? 2 : 1;                             // x
  const int DP = A.dtype == DT_F32 || A.act != ACT_NONE ? 2 : 1;        // du for the layer's gradients
  const int DX = A.dtype == DT_BF16 ? 1 : 2;                            // du for dx
  const int WP = !grouped ? 0 : A.dtype == DT_BF16 ? 1 : 2, per = WP ? WP : 1;
  DuArgs D;
  memset(&D, 0, sizeof(D));
  Carve W{base};
  D.t = A.t; D.m = L.m; D.n = L.n;
  D.mp = mp; D.tp = tp;
  D.rowtiles = mp / 64; D.xtiles = up64(L.n) / 64;
  D.plane_d = up16(A.t) * mp; D.plane_t = up16(L.m) * tp; D.plane_x = up16(L.n) * tp;
  const int64_t plane_w = up16(L.n) * mp, ttiles = tp / 64;
  QGemm gx, gw;
  memset(&gx, 0, sizeof(gx));
  memset(&gw, 0, sizeof(gw));
  q_pairs(gx, per, DX);
  q_pairs(gw, XP, DP);
  const bool sums = A.need_dx && !grouped && L.has_offset();
  D.dmax = W.take<uint32_t>((size_t)A.t * 4);
  D.tmax = W.take<uint32_t>((size_t)L.m * 4);
  D.xmax = W.take<uint32_t>((size_t)L.n * 4);
  D.refs = W.take<uint32_t>((size_t)L.m * 4);
  uint16_t* wt = nullptr;
  float *rowadd = nullptr, *dW = nullptr, *part = nullptr;
  float2* cpart = nullptr;
  size_t ps = 0;
  // rows of the layer whose dW is formed at a time, where it is formed
  const int64_t ldw = (L.n + 3) / 4 * 4, cblocks = (L.n + Q_CONTRACT - 1) / Q_CONTRACT;
  int64_t rows = contract ? L.m : std::max<int64_t>(256, Q_BLOCK_BYTES / (L.n * 4) / 256 * 256);
  rows = std::min(rows, L.m);
  int splits = 1;
  if (A.need_dx) {
    D.d = W.take<uint16_t>((size_t)DX * D.plane_d * 2);
    wt = W.take<uint16_t>((size_t)per * plane_w * 2);
    // (sized without the offset's pointer: room for its sums either way)
    D.rowpart = W.take<float>((size_t)A.t * D.rowtiles * 4);
    rowadd = W.take<float>((size_t)A.t * 4);
    if (!sums) D.rowpart = rowadd = nullptr;
    ps = q_gemm_workspace(L.n, A.t, mp, gx.npairs);
  }
  if (A.need_dlayer) {
    D.dt = W.take<uint16_t>((size_t)DP * D.plane_t * 2);
    D.xt = W.take<uint16_t>((size_t)XP * D.plane_x * 2);
    D.biaspart = W.take<float>((size_t)ttiles * L.m * 4);
    if (contract) {
      splits = q_gemm_splits(L.n, L.m, tp, gw.npairs);
      cpart = W.take<float2>((size_t)splits * L.m * cblocks * sizeof(float2));
    } else {
      dW = W.take<float>((size_t)rows * ldw * 4);
      for (int64_t r0 = 0; r0 < L.m; r0 += rows)
        ps = std::max(ps, q_gemm_workspace(L.n, std::min(rows, L.m - r0), tp, gw.npairs));
    }
  }
  part = W.take<float>(ps);
  if (bytes) *bytes = W.at;
  if (!base) return hipSuccess;

  hipError_t e;
  D.dy = A.dy; D.lddy = A.lddy;
  D.pre = A.pre; D.ldpre = A.ldpre;
  D.x = A.x; D.ldx = A.ldx;
  D.act = A.act; D.dtype = A.dtype;
  D.vec_du = whole_quads(A.dy, A.lddy, A.dtype) && (A.act == ACT_NONE || whole_quads(A.pre, A.ldpre, A.dtype));
  D.vec_x = whole_quads(A.x, A.ldx, A.dtype);
  D.L = L;
  D.want_d = A.need_dx;
  D.want_t = A.need_dlayer;
  D.planes_d = DX; D.planes_t = DP; D.planes_x = XP;
  D.du_blocks = D.rowtiles * ttiles;
  const int64_t x_blocks = A.need_dlayer ? D.xtiles * ttiles : 0;
  const int64_t longest = std::max(std::max(A.t, L.m), L.n);
  hipLaunchKernelGGL(q_grad_init_kernel,
                     dim3((unsigned)std::min<int64_t>(2048, std::max((longest + 255) / 256, grouped ? (L.m + 3) / 4 : 0))),
                     dim3(256), 0, st, D);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(q_grad_scan_kernel, dim3((unsigned)(D.du_blocks + x_blocks)), dim3(256), 0, st, D);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(q_grad_tile_kernel, dim3((unsigned)(D.du_blocks + x_blocks)), dim3(256), 0, st, D);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (sums) {
    hipLaunchKernelGGL(q_grad_rowsum_kernel, dim3((unsigned)((A.t + 255) / 256)), dim3(256), 0, st, D, rowadd);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (A.need_dx) {
    if ((e = unpack_t(L, mp, WP, D.refs, wt, plane_w, st)) != hipSuccess) return e;
    gx.A = wt; gx.planeA = plane_w;
    gx.B = D.d; gx.planeB = D.plane_d;
    gx.M = L.n; gx.N = A.t; gx.K = mp;
    gx.O.y = A.dx; gx.O.ldy = A.lddx;
    gx.O.rowmax = D.dmax;
    gx.O.rowadd = rowadd;
    gx.O.mid = -1;
    gx.O.dtype = A.dtype;
    gx.O.vec = whole_quads(A.dx, A.lddx, A.dtype);
    gx.O.rows = A.t; gx.O.cols = L.n;
    if ((e = launch_q_gemm(gx, part, st)) != hipSuccess) return e;
  }
  if (A.need_dlayer) {
    gw.A = D.xt; gw.planeA = D.plane_x;
    gw.planeB = D.plane_t;
    gw.M = L.n; gw.K = tp;
    gw.O.colmax = D.xmax;
    gw.O.mid = -1;
    gw.O.dtype = DT_F32;
    gw.O.vec = 1;
    gw.O.cols = L.n;
    gw.O.ldy = ldw;
    gw.L = L;
    gw.cpart = cpart; gw.cblocks = cblocks;
    for (int64_t r0 = 0; r0 < L.m; r0 += rows) {
      const int64_t nr = std::min(rows, L.m - r0);
      gw.B = D.dt + r0 * tp;
      gw.N = gw.O.rows = nr;
      gw.O.y = dW;
      gw.O.rowmax = D.tmax + r0;
      gw.row0 = r0;
      if ((e = launch_q_gemm(gw, part, st)) != hipSuccess) return e;
      // d bias rides behind the first block of rows
      const unsigned bias = r0 == 0 ? (unsigned)((L.m + 255) / 256) : 0;
      if (contract)
        hipLaunchKernelGGL(q_contract_finish_kernel, dim3((unsigned)((nr * L.G + 15) / 16) + bias), dim3(256), 0, st, L,
                           cpart, splits, nr, cblocks, r0, A.dscale, A.doffset, D, A.dbias);
      else
        hipLaunchKernelGGL(q_affine_grad_kernel, dim3((unsigned)((nr * L.G + 3) / 4) + bias), dim3(256), 0, st, L, dW,
                           ldw, r0, nr, A.dscale, A.doffset, D, A.dbias);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

size_t q_packed_bytes(const QLayer& L) { return (size_t)L.tiles * L.chunks * 1024; }

hipError_t launch_q_pack(const int32_t* codes, const QLayer& L, void* packed, hipStream_t st) {
  const int64_t total = (int64_t)L.tiles * L.chunks * 64;
  if (total == 0) return hipSuccess;
  hipLaunchKernelGGL(q_pack_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, codes, L,
                     static_cast<uint4*>(packed));
  return hipGetLastError();
}

size_t q_linear_workspace(const QLinearArgs& A) {
  size_t b = 0;
  (void)forward(A, nullptr, &b, nullptr);
  return b;
}
hipError_t launch_q_linear(const QLinearArgs& A, void* ws, hipStream_t st) {
  return forward(A, static_cast<char*>(ws), nullptr, st);
}
size_t q_grad_workspace(const QLinearGrad& A) {
  size_t b = 0;
  (void)backward(A, nullptr, &b, nullptr);
  return b;
}
// Zeros for dx, whose rows may stand apart.
__global__ __launch_bounds__(256) void q_zero_rows_kernel(char* __restrict__ p, int64_t rows, int64_t cols, int64_t ld,
                                                          int es) {
  const int64_t total = rows * cols, step = (int64_t)gridDim.x * 256;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < total; k += step) {
    char* at = p + (k / cols * ld + k % cols) * es;
    if (es == 4) *reinterpret_cast<uint32_t*>(at) = 0;
    else *reinterpret_cast<uint16_t*>(at) = 0;
  }
}
hipError_t launch_q_zero_rows(void* p, int64_t rows, int64_t cols, int64_t ld, int dtype, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>((rows * cols + 255) / 256, 4096);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(q_zero_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, st, static_cast<char*>(p), rows, cols, ld,
                     dtype == DT_F32 ? 4 : 2);
  return hipGetLastError();
}

hipError_t launch_q_grad(const QLinearGrad& A, void* ws, hipStream_t st) {
  return backward(A, static_cast<char*>(ws), nullptr, st);
}

// E8 prefixes: the table of nibbles and the codes' places in it.
//
// Within a shell (points of one norm, in lexicographic order) the negative of
// point k of N is point N - 1 - k, so a point whose negative is among the first
// K codewords too shares one table entry with it.
bool q_e8_tables(const float* cb, int64_t K, uint32_t* lut, uint16_t* map, int* entries, int* pairs) {
  // every codeword's nibbles, 8 + 2 e
  std::vector<uint32_t> nib((size_t)K);
  int32_t odd = 0;
  for (int64_t c = 0; c < K; ++c) {
    int32_t h[8];
    for (int q = 0; q < 8; ++q) {   // (without branches: the host's vectors take it)
      const float x = 2.f * cb[c * 8 + q];
      h[q] = (int32_t)x + 8;
      odd |= ((float)(h[q] - 8) != x) | ((h[q] - 1) & ~15) | (h[q] == 16);
    }
    nib[(size_t)c] = (uint32_t)(h[0] | h[1] << 16 | h[2] << 4 | h[3] << 20 | h[4] << 8 | h[5] << 24 | h[6] << 12) |
                     (uint32_t)h[7] << 28;
  }
  if (odd) return false;
  bool ok = true;
  *pairs = q_e8_pairs(K);
  int64_t pair = 0, lone = 0, s0 = 0;
  for (int h = 0; s0 < K; ++h) {
    const int64_t N = q_e8_shell(h), have = std::min(N, K - s0);
    for (int64_t k = 0; k < have; ++k) {
      const int64_t o = N - 1 - k;
      const uint32_t v = nib[(size_t)(s0 + k)];
      if (o < have && o != k) {
        if (o < k) continue;   // its partner made the entry
        ok &= nib[(size_t)(s0 + o)] == 0x11111110u - v;
        lut[pair] = v;
        map[s0 + k] = (uint16_t)(2 * pair);
        map[s0 + o] = (uint16_t)(2 * pair + 1);
        ++pair;
      } else {
        const int64_t code = 2 * (int64_t)*pairs + lone;
        lut[*pairs + lone] = code & 1 ? 0x11111110u - v : v;
        map[s0 + k] = (uint16_t)code;
        ++lone;
      }
    }
    s0 += N;
  }
  *entries = (int)(*pairs + lone);
  return ok && pair == *pairs && 2 * pair + lone == K;
}

// Points of E8 of squared norm 2 h: 240 times the sum of the cubes of h's divisors.
int64_t q_e8_shell(int h) {
  if (h == 0) return 1;
  int64_t s = 0;
  for (int64_t d = 1; d <= h; ++d)
    if (h % d == 0) s += d * d * d;
  return 240 * s;
}
int q_e8_pairs(int64_t K) {
  int64_t pairs = 0, at = 0;
  for (int h = 0; at < K; ++h) {
    const int64_t N = q_e8_shell(h), have = std::min(N, K - at);
    pairs += h == 0 ? 0 : have == N ? N / 2 : std::max<int64_t>(0, have - N / 2);
    at += N;
  }
  return (int)pairs;
}

}  // namespace mpq
