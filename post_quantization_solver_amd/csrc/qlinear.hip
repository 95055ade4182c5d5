// A solved layer's product and its gradients: packing, operand preparation and
// the order of the launches (qlayer.h; products in qskinny.hip and qgemm.hip).
//
// Many rows: the layer's entries e (one affine per row; exact in 16 bits) or
// its weights a e + o' (column groups; two or three terms) become 16-bit planes
// in the workspace, a block of rows at a time that stays in the last-level
// cache, and the product runs on the matrix cores; the affine, bias,
// activation and residual are its epilogue.
//
// Gradients (codes fixed): du = dy act'(pre);
//   dx = du W: one affine per row: (du a) e + du o', the second a number per
//        row of dx; groups: du times the weights' planes;
//   dW = du^T x, contracted: d scale = sum_j e_ij dW_ij, d offset = sum_j dW_ij
//        over the columns of a group;
//   d bias = sum_t du.
// d scale and d offset are float32 sums: du enters dW as three bfloat16 terms
// (one where it is dy itself), x as its exact terms.  dx is 16 bits wide (or
// float32), so du a is rounded once to its type there (float32: three terms).
#include <string.h>
#include <algorithm>
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
        const int bit = q * bits, hi = bit & 31;
        const uint32_t v = (uint32_t)code << hi;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (bit >> 5 == k) w[k] |= v;
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

// Term p of x as bfloat16: x = sum of the terms, to 2^-8 per term.
__device__ __forceinline__ void bf_terms(float x, uint32_t* b) {
  split3_bf16(x, b[0], b[1], b[2]);
  // an infinite or NaN x stays what it is, alone (inf - inf in a later term is NaN)
  if (!(fabsf(x) <= 3.4028235e38f)) b[1] = b[2] = 0;
}
__device__ __forceinline__ uint32_t widened_or_half(float x, bool half) { return half ? OpF16::bits(x) : f2bf_bits(x); }

// One row of x per workgroup: its 16-bit planes, padded with zeros to Kp
// columns (planes = 0: none), and its sum (optional).
__global__ __launch_bounds__(256) void q_prep_kernel(const void* __restrict__ x, int64_t ldx, int dtype, int64_t n,
                                                     int64_t Kp, uint16_t* __restrict__ out, int64_t plane, int planes,
                                                     bool half, float* __restrict__ sum) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
  float s = 0.f;
  for (int64_t j = threadIdx.x; j < Kp; j += 256) {
    const float v = j < n ? load_as_f32(x, t * ldx + j, dtype) : 0.f;
    s += v;
    if (planes == 1) {
      out[t * Kp + j] = (uint16_t)widened_or_half(v, half);
    } else if (planes > 1) {
      uint32_t b[3];
      bf_terms(v, b);
      for (int p = 0; p < planes; ++p) out[p * plane + t * Kp + j] = (uint16_t)(p == 0 ? b[0] : p == 1 ? b[1] : b[2]);
    }
  }
  if (!sum) return;
  for (int o = 32; o; o >>= 1) s += shfl_xor_f(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) sum[t] = (red[0] + red[1]) + (red[2] + red[3]);
}

// Planes of T terms of the eight values v at step columns.
template <typename T>
__device__ __forceinline__ void weight_terms(const float* v, int planes, v4u* out) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (T::HALF) {
      const uint32_t h = T::pack(v[2 * q], v[2 * q + 1]);
      out[0][q] = h;
      out[1][q] = T::pack(v[2 * q] - T::val(h & 0xffffu), v[2 * q + 1] - T::val(h >> 16));
      out[2][q] = 0u;
    } else {
      uint32_t a[3], b[3];
      bf_terms(v[2 * q], a);
      bf_terms(v[2 * q + 1], b);
#pragma unroll
      for (int p = 0; p < 3; ++p) out[p][q] = pack2(a[p], b[p]);
    }
  }
}

// Eight weights of row i from their entries.
template <typename T>
__device__ __forceinline__ void weights8(const QLayer& L, int64_t i, int64_t j0, v4u e, float mid, float* v) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float x = T::val(q & 1 ? e[q >> 1] >> 16 : e[q >> 1] & 0xffffu);
    const int64_t j = min(j0 + q, L.n - 1);
    const int64_t g = i * L.G + (L.G > 1 ? j / L.group : 0);
    const float a = L.scale[g];
    v[q] = j0 + q < L.n ? fmaf(a, x, fmaf(a, mid, L.offset ? L.offset[g] : 0.f)) : 0.f;
  }
}

// Rows tile0 * 16 .. of the layer as planes of Kp columns: entries (planes = 0),
// or weights in `planes` terms.  A wave per chunk of a tile.
template <int FMT, typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void q_unpack_kernel(QLayer L, int tile0, int tiles, int64_t Kp, int planes,
                                                              uint16_t* __restrict__ out, int64_t plane) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int lane = threadIdx.x & 63, wave = wave_id();
  q_lut_fill<FMT, T>(L, lds, 64 * WAVES);
  __syncthreads();
  const float mid = q_centre(L);
  const int64_t total = (int64_t)tiles * L.chunks;
  for (int64_t w = (int64_t)blockIdx.x * WAVES + wave; w < total; w += (int64_t)gridDim.x * WAVES) {
    const int tl = (int)(w / L.chunks), c = (int)(w - (int64_t)tl * L.chunks);
    const uint4 code = L.packed[((size_t)(tile0 + tl) * L.chunks + c) * 64 + lane];
    const int64_t row = tl * 16 + (lane & 15), i = (int64_t)tile0 * 16 + row;
#pragma unroll
    for (int s = 0; s < q_steps(FMT); ++s) {
      const int64_t j0 = (((int64_t)c * q_steps(FMT) + s) * 4 + (lane >> 4)) * 8;
      v4u e = q_decode<FMT, T>(L, lds, code, s);
      if (i >= L.m || j0 >= Kp) continue;
      uint16_t* dst = out + row * Kp + j0;
      if (planes == 0) {
        // columns past the last hold zero, whatever their codes
        if (j0 + 8 > L.n) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (j0 + q >= L.n) e[q >> 1] &= q & 1 ? 0xffffu : 0xffff0000u;
        }
        *reinterpret_cast<v4u*>(dst) = e;
      } else {
        float v[8];
        v4u o[3];
        weights8<T>(L, i, j0, e, mid, v);
        weight_terms<T>(v, planes, o);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          if (p < planes) *reinterpret_cast<v4u*>(dst + p * plane) = o[p];
      }
    }
  }
}

// The transpose: plane rows are the layer's columns, mp (m padded with zeros
// to 64) entries or weights each.  A workgroup unpacks 16 WAVES rows of one
// chunk, 32 columns at a time, through LDS.
template <int FMT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void q_unpack_t_kernel(QLayer L, int64_t mp, int planes,
                                                                uint16_t* __restrict__ out, int64_t plane,
                                                                int lut_words) {
  using T = OpBf16;
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int ROWS = 16 * WAVES;
  uint16_t* tl = reinterpret_cast<uint16_t*>(lds + lut_words);   // 32 columns x ROWS
  const int lane = threadIdx.x & 63, wave = wave_id();
  q_lut_fill<FMT, T>(L, lds, 64 * WAVES);
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
    const int64_t i = tile * 16 + (lane & 15);
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
      v4u e = q_decode<FMT, T>(L, lds, cs, 0);
      const int64_t j0 = (((int64_t)c * q_steps(FMT) + s) * 4 + (lane >> 4)) * 8;
      v4u o[3];
      if (i >= L.m) e = (v4u){0u, 0u, 0u, 0u};
      o[0] = e;
      if (planes > 0) {
        float v[8];
        weights8<T>(L, min(i, L.m - 1), j0, e, mid, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = i < L.m ? v[q] : 0.f;
        weight_terms<T>(v, planes, o);
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        if (p >= (planes > 0 ? planes : 1)) break;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          tl[((lane >> 4) * 8 + q) * ROWS + wave * 16 + (lane & 15)] =
              (uint16_t)(q & 1 ? o[p][q >> 1] >> 16 : o[p][q >> 1] & 0xffffu);
        __syncthreads();
        constexpr int PIECES = ROWS / 8;
        for (int k = threadIdx.x; k < 32 * PIECES; k += 64 * WAVES) {
          const int col = k / PIECES, piece = k - col * PIECES;
          const int64_t j = ((int64_t)c * q_steps(FMT) + s) * 32 + col;
          const int64_t r = strip * ROWS + piece * 8;
          if (j < L.n && r < mp)
            *reinterpret_cast<v4u*>(out + p * plane + j * mp + r) =
                *reinterpret_cast<const v4u*>(tl + col * ROWS + piece * 8);
        }
        __syncthreads();
      }
    }
  }
}

// Bfloat16 planes of x^T: n rows of tp (t padded with zeros to 64).
__global__ __launch_bounds__(256) void q_transpose_kernel(const void* __restrict__ x, int64_t ldx, int dtype, int64_t t,
                                                          int64_t n, int64_t tp, int planes,
                                                          uint16_t* __restrict__ out, int64_t plane) {
  __shared__ float tl[64][65];
  const int64_t j0 = (int64_t)blockIdx.x * 64, t0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  for (int y = ty; y < 64; y += 4)
    tl[y][tx] = t0 + y < t && j0 + tx < n ? load_as_f32(x, (t0 + y) * ldx + j0 + tx, dtype) : 0.f;
  __syncthreads();
  for (int y = ty; y < 64; y += 4) {
    if (j0 + y >= n) break;
    uint32_t b[3];
    bf_terms(tl[tx][y], b);
    for (int p = 0; p < planes; ++p)
      out[p * plane + (j0 + y) * tp + t0 + tx] = (uint16_t)(p == 0 ? b[0] : p == 1 ? b[1] : b[2]);
  }
}

struct DuArgs {
  const void* dy; int64_t lddy;
  const void* pre; int64_t ldpre;
  int act, dtype;
  int64_t t, m;
  // (du a) or du, t rows of mp
  uint16_t* d; int64_t plane_d, mp; int planes_d;
  const float* scale;                 // per row of the layer, or nullptr
  const float* offset;                // with scale
  const float* levels; int mid;
  float* rowpart; int64_t rowtiles;   // t x rowtiles: sums of du o' over 64 columns (nullptr: none)
  // du^T, m rows of tp
  uint16_t* dt; int64_t plane_t, tp; int planes_t;
  float* biaspart;                    // (tp / 64) x m: sums of du over 64 rows
};

// A 64 x 64 tile of du: its planes, its transpose's planes, its row and column sums.
__global__ __launch_bounds__(256) void q_du_kernel(DuArgs A) {
  __shared__ float tl[64][65];
  const int64_t i0 = (int64_t)blockIdx.x * 64, t0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int64_t i = i0 + tx;
  float a = 1.f, o = 0.f;
  if (A.scale && i < A.m) {
    a = A.scale[i];
    o = fmaf(a, A.mid >= 0 ? A.levels[A.mid] : 0.f, A.offset ? A.offset[i] : 0.f);
  }
  for (int y = ty; y < 64; y += 4) {
    float v = 0.f;
    if (t0 + y < A.t && i < A.m) {
      v = load_as_f32(A.dy, (t0 + y) * A.lddy + i, A.dtype);
      if (A.act != ACT_NONE) v *= act_slope(A.act, load_as_f32(A.pre, (t0 + y) * A.ldpre + i, A.dtype));
    }
    tl[y][tx] = v;
    if (A.d && t0 + y < A.t && i < A.mp) {
      uint32_t b[3];
      bf_terms(A.scale ? v * a : v, b);
      for (int p = 0; p < A.planes_d; ++p)
        A.d[p * A.plane_d + (t0 + y) * A.mp + i] = (uint16_t)(p == 0 ? b[0] : p == 1 ? b[1] : b[2]);
    }
    if (A.rowpart) {
      float s = v * o;
      for (int k = 32; k; k >>= 1) s += shfl_xor_f(s, k);
      if (tx == 0 && t0 + y < A.t) A.rowpart[(t0 + y) * A.rowtiles + blockIdx.x] = s;
    }
  }
  __syncthreads();
  if (!A.dt) return;
  for (int y = ty; y < 64; y += 4) {
    if (i0 + y >= A.m) break;
    const float v = tl[tx][y];
    uint32_t b[3];
    bf_terms(v, b);
    for (int p = 0; p < A.planes_t; ++p)
      A.dt[p * A.plane_t + (i0 + y) * A.tp + t0 + tx] = (uint16_t)(p == 0 ? b[0] : p == 1 ? b[1] : b[2]);
    float s = v;
    for (int k = 32; k; k >>= 1) s += shfl_xor_f(s, k);
    if (tx == 0) A.biaspart[blockIdx.y * A.m + i0 + y] = s;
  }
}

// out[r] = sum of part[r * ld + k * step], k < count, in order, in float64.
__global__ __launch_bounds__(256) void q_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t ld,
                                                    int64_t step, int64_t count, float* __restrict__ out) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  double s = 0.0;
  for (int64_t k = 0; k < count; ++k) s += (double)part[r * ld + k * step];
  out[r] = (float)s;
}

// d scale and d offset of `rows` rows from row0 on: a wave per (row, group).
__global__ __launch_bounds__(256) void q_affine_grad_kernel(QLayer L, const float* __restrict__ dW, int64_t ldw,
                                                            int64_t row0, int64_t rows, float* __restrict__ dscale,
                                                            float* __restrict__ doffset) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= rows * L.G) return;
  const int64_t row = w / L.G, g = w - row * L.G, i = row0 + row;
  const int64_t j0 = g * L.group, j1 = min(L.n, j0 + L.group);
  const int steps = q_steps(L.fmt);
  const uint16_t* codes = reinterpret_cast<const uint16_t*>(L.packed);
  double se = 0.0, s1 = 0.0;
  for (int64_t j = j0 + lane; j < j1; j += 64) {
    const float d = dW[row * ldw + j];
    // the weight's place in the packed tile
    const int64_t blk = j >> 3, c = blk / (4 * steps);
    const int kb = (int)(blk & 3), s = (int)(blk - c * 4 * steps) >> 2, q = (int)(j & 7);
    const size_t at = (((size_t)(i >> 4) * L.chunks + c) * 64 + kb * 16 + (i & 15)) * 8;   // 16-bit words
    float e;
    if (L.fmt == QF_NIB) {
      e = L.levels[(codes[at + s * 2 + (q >> 2)] >> (4 * (q & 3))) & 15];
    } else if (L.fmt == QF_BYTE) {
      e = L.levels[(codes[at + s * 4 + (q >> 1)] >> (8 * (q & 1))) & 255];
    } else if (L.fmt == QF_E8) {
      const int code = codes[at + s];
      const uint32_t v = L.lut[max(code >> 1, code - L.pairs)] ^ (code & 1 ? 0x88888888u : 0u);
      const uint32_t nib = v >> (4 * (q < 4 ? 2 * q : 2 * q - 7));
      e = 0.5f * (float)(nib & 7u) * (nib & 8u ? -1.f : 1.f);
    } else {
      e = L.e32[(size_t)codes[at + s] * 8 + q];
    }
    se += (double)(e * d);
    s1 += (double)d;
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
hipError_t unpack(const QLayer& L, int tile0, int tiles, int64_t Kp, int planes, uint16_t* out, int64_t plane,
                  hipStream_t st) {
  const size_t shared = (size_t)q_lut_words(L.fmt, (L.lut_entries + 3) / 4 * 4) * 4;
  const int64_t waves = (int64_t)tiles * L.chunks;
  auto grid = [&](int per, int most) { return dim3((unsigned)std::min<int64_t>((waves + per - 1) / per, most)); };
  switch (L.fmt) {
    case QF_NIB:
      hipLaunchKernelGGL((q_unpack_kernel<QF_NIB, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, out, plane);
      break;
    case QF_BYTE:
      hipLaunchKernelGGL((q_unpack_kernel<QF_BYTE, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, out, plane);
      break;
    case QF_E8:   // the table fills a CU's LDS: one workgroup of 16 waves each
      hipLaunchKernelGGL((q_unpack_kernel<QF_E8, T, 16>), grid(16, 256), dim3(1024), shared, st, L, tile0, tiles, Kp,
                         planes, out, plane);
      break;
    default:
      hipLaunchKernelGGL((q_unpack_kernel<QF_VEC, T, 4>), grid(4, 2048), dim3(256), shared, st, L, tile0, tiles, Kp,
                         planes, out, plane);
  }
  return hipGetLastError();
}

hipError_t unpack_t(const QLayer& L, int64_t mp, int planes, uint16_t* out, int64_t plane, hipStream_t st) {
  const int lut = q_lut_words(L.fmt, (L.lut_entries + 3) / 4 * 4);
  auto go = [&](auto kernel, int waves, int most) {
    const int64_t total = (mp + 16 * waves - 1) / (16 * waves) * L.chunks;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(total, most)), dim3(64 * waves),
                       (size_t)lut * 4 + (size_t)32 * 16 * waves * 2, st, L, mp, planes, out, plane, lut);
  };
  switch (L.fmt) {
    case QF_NIB: go(q_unpack_t_kernel<QF_NIB, 4>, 4, 2048); break;
    case QF_BYTE: go(q_unpack_t_kernel<QF_BYTE, 4>, 4, 2048); break;
    case QF_E8: go(q_unpack_t_kernel<QF_E8, 8>, 8, 256); break;
    default: go(q_unpack_t_kernel<QF_VEC, 4>, 4, 2048); break;
  }
  return hipGetLastError();
}

// The operand planes of x for the forward product: x itself where its rows
// are 16-bit, 16-byte aligned and whole steps, else padded copies.
struct XPlan {
  bool direct, half;
  int planes;
  int64_t Kp;
};
XPlan x_plan(const QLinearArgs& A, bool skinny) {
  XPlan P;
  P.half = A.dtype == DT_F16;
  P.planes = A.dtype == DT_F32 ? 3 : 1;
  P.Kp = up64(A.L.n);
  const bool aligned = reinterpret_cast<uintptr_t>(A.x) % 16 == 0 && A.ldx % 8 == 0 && A.ldx <= (1 << 20);
  P.direct = P.planes == 1 && aligned && A.L.n % (skinny ? 8 : 64) == 0;
  return P;
}

// Token counts from which the unpacked product is used.  (One affine per row and groups of whole chunks; other
// groups always unpack.)
int64_t skinny_tokens(const QLayer&) { return 128; }

bool use_skinny(const QLinearArgs& A) { return q_skinny_ok(A.L) && A.t <= skinny_tokens(A.L); }

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

// Forward: lays out the workspace and, with a base, launches.
hipError_t forward(const QLinearArgs& A, char* base, size_t* bytes, hipStream_t st) {
  const QLayer& L = A.L;
  const bool skinny = use_skinny(A);
  const XPlan P = x_plan(A, skinny);
  Carve W{base};
  // (the layout does not depend on x's alignment: the caller sizes it without x)
  const int64_t plane = A.t * P.Kp;
  uint16_t* xp = W.take<uint16_t>((size_t)P.planes * plane * 2);
  float* xs = W.take<float>((size_t)A.t * 4);
  const bool grouped = L.G > 1, sums = !skinny && !grouped && L.has_offset();
  const int WP = !grouped ? 0 : A.dtype == DT_F32 ? 3 : 2;   // terms of a weight (0: entries)
  const int per = WP ? WP : 1;
  int64_t rows = std::max<int64_t>(256, Q_BLOCK_BYTES / (per * P.Kp * 2) / 256 * 256);
  rows = std::min(rows, (int64_t)L.tiles * 16);
  QGemm g;
  memset(&g, 0, sizeof(g));
  if (WP) q_pairs(g, WP, P.planes); else q_pairs(g, 1, P.planes);
  uint16_t* wp = nullptr;
  float* part = nullptr;
  if (!skinny) {
    wp = W.take<uint16_t>((size_t)per * rows * P.Kp * 2);
    size_t ps = 0;
    for (int64_t r0 = 0; r0 < L.m; r0 += rows)
      ps = std::max(ps, q_gemm_workspace(std::min(rows, L.m - r0), A.t, P.Kp, g.npairs));
    part = W.take<float>(ps);
  }
  if (bytes) *bytes = W.at;
  if (!base) return hipSuccess;

  hipError_t e;
  if (!P.direct || sums) {
    hipLaunchKernelGGL(q_prep_kernel, dim3((unsigned)A.t), dim3(256), 0, st, A.x, A.ldx, A.dtype, L.n, P.Kp, xp, plane,
                       P.direct ? 0 : P.planes, P.half, sums ? xs : nullptr);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const uint16_t* x = P.direct ? static_cast<const uint16_t*>(A.x) : xp;
  const int64_t ldx = P.direct ? A.ldx : P.Kp;
  QOut O;
  memset(&O, 0, sizeof(O));
  O.y = A.y; O.ldy = A.ldy;
  O.pre = A.pre; O.ldpre = A.ldpre;
  O.res = A.res; O.ldres = A.ldres;
  O.bias = A.bias;
  O.act = A.act;
  O.dtype = A.dtype;
  O.mid = -1;
  O.rows = A.t;
  O.cols = L.m;
  const uintptr_t quad = A.dtype == DT_F32 ? 16 : 8;
  auto whole = [&](const void* p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % quad == 0 && ld % 4 == 0);
  };
  O.vec = whole(A.y, A.ldy) && whole(A.pre, A.ldpre) && whole(A.res, A.ldres);
  if (skinny)
    return launch_q_skinny(L, x, ldx, plane, (int)(P.direct ? L.n / 8 : P.Kp / 8), A.t, P.planes, P.half, O, st);
  const int es = A.dtype == DT_F32 ? 4 : 2;
  for (int64_t r0 = 0; r0 < L.m; r0 += rows) {
    const int64_t nr = std::min(rows, L.m - r0);
    const int tiles = (int)((nr + 15) / 16);
    e = P.half ? unpack<OpF16>(L, (int)(r0 / 16), tiles, P.Kp, WP, wp, rows * P.Kp, st)
               : unpack<OpBf16>(L, (int)(r0 / 16), tiles, P.Kp, WP, wp, rows * P.Kp, st);
    if (e != hipSuccess) return e;
    g.A = wp; g.lda = P.Kp; g.planeA = rows * P.Kp;
    g.B = x; g.ldb = ldx; g.planeB = plane;
    g.M = nr; g.N = A.t; g.K = P.Kp;
    g.half = P.half;
    g.O = O;
    g.O.cols = nr;
    g.O.y = static_cast<char*>(A.y) + r0 * es;
    if (A.pre) g.O.pre = static_cast<char*>(A.pre) + r0 * es;
    if (A.res) g.O.res = static_cast<const char*>(A.res) + r0 * es;
    if (A.bias) g.O.bias = A.bias + r0;
    if (!grouped) {
      g.O.colscale = L.scale + r0;
      g.O.coloff = L.offset ? L.offset + r0 : nullptr;
      g.O.rowadd = sums ? xs : nullptr;
      g.O.levels = L.levels;
      g.O.mid = L.fmt == QF_NIB || L.fmt == QF_BYTE ? L.K / 2 : -1;
    }
    if ((e = launch_q_gemm(g, part, st)) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t backward(const QLinearGrad& A, char* base, size_t* bytes, hipStream_t st) {
  const QLayer& L = A.L;
  const bool grouped = L.G > 1;
  const int64_t mp = up64(L.m), tp = up64(A.t);
  const int XP = A.dtype == DT_F32 ? 3 : A.dtype == DT_F16 ? 2 : 1;             // x, exactly
  const int DP = A.act == ACT_NONE ? XP : 3;                                    // du for dW: exactly, or 24 bits
  const int DX = A.dtype == DT_F32 ? 3 : A.dtype == DT_F16 ? 2 : 1;             // du (a) for dx
  const int WP = !grouped ? 0 : A.dtype == DT_F32 ? 3 : 2, per = WP ? WP : 1;   // weights for dx
  Carve W{base};
  const int64_t plane_d = A.t * mp, plane_t = L.m * tp, plane_w = L.n * mp, plane_x = L.n * tp;
  const int64_t rowtiles = mp / 64, ttiles = tp / 64;
  uint16_t *d = nullptr, *dt = nullptr, *wt = nullptr, *xt = nullptr;
  float *rowpart = nullptr, *rowadd = nullptr, *biaspart = nullptr, *dW = nullptr, *part = nullptr;
  QGemm gx, gw;
  memset(&gx, 0, sizeof(gx));
  memset(&gw, 0, sizeof(gw));
  q_pairs(gx, per, DX);
  q_pairs(gw, XP, DP);
  const bool sums = A.need_dx && !grouped && L.has_offset();
  // rows of the layer whose dW is formed at a time
  int64_t rows = std::max<int64_t>(256, Q_BLOCK_BYTES / (L.n * 4) / 256 * 256);
  rows = std::min(rows, L.m);
  const int64_t ldw = (L.n + 3) / 4 * 4;
  size_t ps = 0;
  if (A.need_dx) {
    d = W.take<uint16_t>((size_t)DX * plane_d * 2);
    wt = W.take<uint16_t>((size_t)per * plane_w * 2);
    // (sized without the offset's pointer: room for its sums either way)
    rowpart = W.take<float>((size_t)A.t * rowtiles * 4);
    rowadd = W.take<float>((size_t)A.t * 4);
    if (!sums) rowpart = rowadd = nullptr;
    ps = q_gemm_workspace(L.n, A.t, mp, gx.npairs);
  }
  if (A.need_dlayer) {
    dt = W.take<uint16_t>((size_t)DP * plane_t * 2);
    xt = W.take<uint16_t>((size_t)XP * plane_x * 2);
    biaspart = W.take<float>((size_t)ttiles * L.m * 4);
    dW = W.take<float>((size_t)rows * ldw * 4);
    for (int64_t r0 = 0; r0 < L.m; r0 += rows)
      ps = std::max(ps, q_gemm_workspace(L.n, std::min(rows, L.m - r0), tp, gw.npairs));
  }
  part = W.take<float>(ps);
  if (bytes) *bytes = W.at;
  if (!base) return hipSuccess;

  hipError_t e;
  DuArgs D;
  memset(&D, 0, sizeof(D));
  D.dy = A.dy; D.lddy = A.lddy;
  D.pre = A.pre; D.ldpre = A.ldpre;
  D.act = A.act; D.dtype = A.dtype;
  D.t = A.t; D.m = L.m;
  D.d = d; D.plane_d = plane_d; D.mp = mp; D.planes_d = DX;
  D.mid = L.fmt == QF_NIB || L.fmt == QF_BYTE ? L.K / 2 : -1;
  D.levels = L.levels;
  if (A.need_dx && !grouped) {
    D.scale = L.scale;
    D.offset = L.offset;
  }
  D.rowpart = rowpart; D.rowtiles = rowtiles;
  D.dt = dt; D.plane_t = plane_t; D.tp = tp; D.planes_t = DP;
  D.biaspart = biaspart;
  hipLaunchKernelGGL(q_du_kernel, dim3((unsigned)rowtiles, (unsigned)ttiles), dim3(256), 0, st, D);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const uintptr_t quad = A.dtype == DT_F32 ? 16 : 8;
  if (A.need_dx) {
    if (sums) {
      hipLaunchKernelGGL(q_sum_kernel, dim3((unsigned)((A.t + 255) / 256)), dim3(256), 0, st, rowpart, A.t, rowtiles,
                         (int64_t)1, rowtiles, rowadd);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if ((e = unpack_t(L, mp, WP, wt, plane_w, st)) != hipSuccess) return e;
    gx.A = wt; gx.lda = mp; gx.planeA = plane_w;
    gx.B = d; gx.ldb = mp; gx.planeB = plane_d;
    gx.M = L.n; gx.N = A.t; gx.K = mp;
    gx.O.y = A.dx; gx.O.ldy = A.lddx;
    gx.O.rowadd = rowadd;
    gx.O.mid = -1;
    gx.O.dtype = A.dtype;
    gx.O.vec = reinterpret_cast<uintptr_t>(A.dx) % quad == 0 && A.lddx % 4 == 0;
    gx.O.rows = A.t; gx.O.cols = L.n;
    if ((e = launch_q_gemm(gx, part, st)) != hipSuccess) return e;
  }
  if (A.need_dlayer) {
    hipLaunchKernelGGL(q_transpose_kernel, dim3((unsigned)((L.n + 63) / 64), (unsigned)ttiles), dim3(256), 0, st, A.x,
                       A.ldx, A.dtype, A.t, L.n, tp, XP, xt, plane_x);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(q_sum_kernel, dim3((unsigned)((L.m + 255) / 256)), dim3(256), 0, st, biaspart, L.m, (int64_t)1,
                       L.m, ttiles, A.dbias);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    for (int64_t r0 = 0; r0 < L.m; r0 += rows) {
      const int64_t nr = std::min(rows, L.m - r0);
      gw.A = xt; gw.lda = tp; gw.planeA = plane_x;
      gw.B = dt + r0 * tp; gw.ldb = tp; gw.planeB = plane_t;
      gw.M = L.n; gw.N = nr; gw.K = tp;
      gw.O.y = dW; gw.O.ldy = ldw;
      gw.O.mid = -1;
      gw.O.dtype = DT_F32;
      gw.O.vec = 1;
      gw.O.rows = nr; gw.O.cols = L.n;
      if ((e = launch_q_gemm(gw, part, st)) != hipSuccess) return e;
      hipLaunchKernelGGL(q_affine_grad_kernel, dim3((unsigned)((nr * L.G + 3) / 4)), dim3(256), 0, st, L, dW, ldw, r0,
                         nr, A.dscale, A.doffset);
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
hipError_t launch_q_grad(const QLinearGrad& A, void* ws, hipStream_t st) {
  return backward(A, static_cast<char*>(ws), nullptr, st);
}

// E8 prefixes: the sign-magnitude table and the codes' places in it.
//
// Within a shell (points of one norm, in lexicographic order) the negative of
// point k of N is point N - 1 - k, so a point whose negative is among the first
// K codewords too shares one table entry with it.
bool q_e8_tables(const float* cb, int64_t K, uint32_t* lut, uint16_t* map, int* entries, int* pairs) {
  auto nibbles = [&](int64_t c, uint32_t* v) {
    *v = 0;
    for (int q = 0; q < 8; ++q) {
      const float x = cb[c * 8 + q];
      const int h = (int)(2.f * (x < 0 ? -x : x));
      if (h > 7 || 0.5f * h != (x < 0 ? -x : x)) return false;
      *v |= (uint32_t)(h | (x < 0 ? 8 : 0)) << (4 * (q < 4 ? 2 * q : 2 * q - 7));
    }
    return true;
  };
  auto norm = [&](int64_t c) {
    float s = 0.f;
    for (int q = 0; q < 8; ++q) s += cb[c * 8 + q] * cb[c * 8 + q];
    return s;
  };
  *pairs = q_e8_pairs(K);
  int64_t pair = 0, lone = 0;
  for (int64_t s0 = 0; s0 < K;) {
    int64_t s1 = s0 + 1;
    while (s1 < K && norm(s1) == norm(s0)) ++s1;
    const int64_t N = q_e8_shell((int)(norm(s0) / 2.f)), have = s1 - s0;
    for (int64_t k = 0; k < have; ++k) {
      const int64_t o = N - 1 - k;
      uint32_t v;
      if (!nibbles(s0 + k, &v)) return false;
      if (o < have && o != k) {
        if (o < k) continue;   // its partner made the entry
        for (int q = 0; q < 8; ++q)
          if (cb[(s0 + k) * 8 + q] != -cb[(s0 + o) * 8 + q]) return false;
        lut[pair] = v;
        map[s0 + k] = (uint16_t)(2 * pair);
        map[s0 + o] = (uint16_t)(2 * pair + 1);
        ++pair;
      } else {
        const int64_t code = 2 * (int64_t)*pairs + lone;
        lut[*pairs + lone] = code & 1 ? v ^ 0x88888888u : v;
        map[s0 + k] = (uint16_t)code;
        ++lone;
      }
    }
    s0 = s1;
  }
  *entries = (int)(*pairs + lone);
  return pair == *pairs && 2 * pair + lone == K;
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
