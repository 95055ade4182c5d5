// Packed codes of a solved layer and what the kernels that read them share.
//
// A layer's m x n weights are W[i][j] = a e + o with base entries e of a
// codebook.  Codes are packed in tiles of 16 rows: chunk c of a tile holds
// q_steps(f) * 32 columns as 64 lanes x 16 bytes, lane l holding row l % 16 and,
// for step s, columns s * 32 + (l / 16) * 8 .. + 7 of the chunk.  One wave load
// is 1 KB of contiguous memory, and what lane l decodes for step s is its
// operand of v_mfma_f32_16x16x32 as it stands; a row's four lanes of a step
// cover 64 consecutive bytes of 16-bit activations or unpacked entries.
//
// d = 1: entries are taken about the middle level, e - levels[K / 2], so that
// the sums over a grid 0 .. K - 1 do not carry a large common part that the
// offset takes off again; o' = o + a levels[K / 2].  A step's eight 4-bit codes
// are stored with code 2 p in nibble p and code 2 p + 1 in nibble p + 4, its
// 8-bit codes with code 2 p in byte p and code 2 p + 1 in byte p + 2 (of a word
// of four): a pair is 16 bits apart, where a pair of 16-bit values wants it.
#pragma once
#include "mpq_device.h"
#include "internal.h"

namespace mpq {

enum QFormat : int {
  QF_NIB = 0,    // d = 1, K <= 16: 4 bits a weight
  QF_BYTE = 1,   // d = 1, K <= 64: 8 bits a weight
  QF_E8 = 2,     // the first K points of E8: 16 bits per 8 weights, re-indexed (see q_e8_tables)
  QF_VEC = 3,    // other d = 8 codebooks: the codes, 16 bits per 8 weights
};
__host__ __device__ constexpr int q_steps(int f) { return f == QF_NIB ? 4 : f == QF_BYTE ? 2 : 8; }
__host__ __device__ constexpr int q_chunk(int f) { return q_steps(f) * 32; }

// Dwords of the decoder's LDS table.
inline int q_lut_words(int f, int entries) { return f == QF_NIB ? 256 : f == QF_BYTE ? 4096 : f == QF_E8 ? entries : 0; }

struct QLayer {
  int fmt;
  int64_t m, n;
  int tiles, chunks;
  const uint4* packed;
  const float* scale;    // m x G
  const float* offset;   // m x G, or nullptr: zero
  int64_t group; int G;  // columns per affine group (n: one per row)
  const float* levels;   // d = 1
  bool uniform;          // d = 1: levels[q] = levels[0] + q (levels[1] - levels[0]), exactly
  int K;
  const uint32_t* lut;   // QF_E8: nibbles 8 + 2 e, coordinate 2 p in nibble p, 2 p + 1 in nibble p + 4
  const uint16_t* map;   // QF_E8: code -> packed code
  int lut_entries, pairs;
  const float* e32;      // d = 8: K x 8
  bool has_offset() const { return offset != nullptr || fmt == QF_NIB || fmt == QF_BYTE; }
};

#ifdef __HIPCC__
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// The matrix cores' 16-bit operand types.
struct OpBf16 {
  static constexpr bool HALF = false;
  __device__ static v4f mfma(v4u a, v4u b, v4f c) { return mfma_bf16_16x16x32(a, b, c); }
  __device__ static uint32_t bits(float x) { return f2bf_bits(x); }
  __device__ static float val(uint32_t b) { return bf_bits2f(b & 0xffffu); }
  __device__ static uint32_t pack(float x, float y) { return f2bf_pack(x, y); }
  static constexpr uint32_t ONES = 0x3f803f80u;
};
struct OpF16 {
  static constexpr bool HALF = true;
  __device__ static v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  __device__ static uint32_t bits(float x) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x); }
  __device__ static float val(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }
  __device__ static uint32_t pack(float x, float y) {
    v2h v = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
  static constexpr uint32_t ONES = 0x3c003c00u;
};

__device__ __forceinline__ float q_centre(const QLayer& L) {
  return L.fmt == QF_NIB || L.fmt == QF_BYTE ? L.levels[L.K / 2] : 0.f;
}

// 16 bytes a lane from src (this lane's) to dst (the wave's, 1 KB), past the registers.
typedef __attribute__((address_space(3))) void* q_lds_ptr;
__device__ __forceinline__ void q_load_lds(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (q_lds_ptr)dst, 16, 0, 0);
}
// The operand of s_waitcnt: at most n loads on their way, and no LDS operation.
constexpr int q_waitcnt(int n) { return (n & 15) | 7 << 4 | (n >> 4) << 14; }

// Fills the decoder's LDS table (every thread of the workgroup; the caller
// synchronizes, for E8 after a wait for the loads: q_lut_wait).
template <int FMT, typename T>
__device__ __forceinline__ void q_lut_fill(const QLayer& L, uint32_t* lut, int nthreads) {
  const int t = threadIdx.x;
  if constexpr (FMT == QF_E8) {
    const int quads = (L.lut_entries + 3) / 4;   // the table is padded to 16 bytes
    for (int i = t; i < quads; i += nthreads)
      q_load_lds(reinterpret_cast<const uint4*>(L.lut) + i, reinterpret_cast<uint4*>(lut) + (i & ~63));
  } else if constexpr (FMT == QF_NIB || FMT == QF_BYTE) {
    constexpr int BITS = FMT == QF_NIB ? 4 : 6;
    const float mid = q_centre(L);
    for (int i = t; i < 1 << (2 * BITS); i += nthreads) {
      const int lo = i & ((1 << BITS) - 1), hi = i >> BITS;
      lut[i] = T::pack(L.levels[lo < L.K ? lo : 0] - mid, L.levels[hi < L.K ? hi : 0] - mid);
    }
  }
}

// Waits for the table's loads; `after` loads went out behind them.
template <int AFTER>
__device__ __forceinline__ void q_lut_wait() {
  static_assert(AFTER < 64, "the counter has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(q_waitcnt(AFTER));
  asm volatile("" ::: "memory");
}

// The table's nibbles of a packed E8 code (its low 16 bits): 2 i + sign for the
// i-th of `pairs` points whose negative is in the codebook too, pairs + i for
// entry i beyond them; either way the entry is max(code / 2, code - pairs), and
// an odd code negates it (a lone entry with an odd code is stored negated).
// Nibbles are 1 to 15, so that 16 - v goes through all eight without a carry.
__device__ __forceinline__ uint32_t q_e8_nibbles(const QLayer& L, const uint32_t* lut, uint32_t word) {
  const uint32_t code = word & 0xffffu;
  const uint32_t v = lut[max((int)(code >> 1), (int)code - L.pairs)];
  const uint32_t odd = (uint32_t)((int)(word << 31) >> 31);
  return (v ^ odd) + (odd & 0x11111111u);
}

// The nibbles as entries, or, in bfloat16, lifted: 64 + q / 2 (the entry and 68).
template <typename T>
__device__ __forceinline__ v4u q_e8_entries(uint32_t v) {
  v4u r;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t q = (v >> (4 * b)) & 0x000f000fu;
    if constexpr (T::HALF) {   // 512 + q / 2 is 0x6000 | q
      r[b] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, q | 0x60006000u) +
                                              (v2h){(_Float16)-516.f, (_Float16)-516.f});
    } else {                   // 64 + q / 2 is 0x4280 | q
      const uint32_t u = q | 0x42804280u;
      r[b] = __builtin_amdgcn_perm(__float_as_uint(__uint_as_float(u & 0xffff0000u) - 68.f),
                                   __float_as_uint(__uint_as_float(u << 16) - 68.f), 0x07060302u);
    }
  }
  return r;
}
__device__ __forceinline__ v4u q_e8_lifted(uint32_t v) {
  v4u r;
#pragma unroll
  for (int b = 0; b < 4; ++b) r[b] = ((v >> (4 * b)) & 0x000f000fu) | 0x42804280u;
  return r;
}

// The eight entries of step s from a lane's 16 bytes of codes.
template <int FMT, typename T>
__device__ __forceinline__ v4u q_decode(const QLayer& L, const uint32_t* lut, const uint4& c, int s) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  v4u r;
  if constexpr (FMT == QF_NIB) {
#pragma unroll
    for (int b = 0; b < 4; ++b) r[b] = lut[((w[s] >> (4 * b)) & 15u) | ((w[s] >> (4 * b + 12)) & 240u)];
  } else if constexpr (FMT == QF_BYTE) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t h = w[2 * s + (b >> 1)] >> (8 * (b & 1));
      r[b] = lut[(h & 63u) | ((h >> 10) & 0xfc0u)];
    }
  } else if constexpr (FMT == QF_E8) {
    r = q_e8_entries<T>(q_e8_nibbles(L, lut, w[s >> 1] >> (16 * (s & 1))));
  } else {
    const uint32_t code = (w[s >> 1] >> (16 * (s & 1))) & 0xffffu;
    const float4* e = reinterpret_cast<const float4*>(L.e32 + (size_t)code * 8);
    const float4 a = e[0], b = e[1];
    r[0] = T::pack(a.x, a.y);
    r[1] = T::pack(a.z, a.w);
    r[2] = T::pack(b.x, b.y);
    r[3] = T::pack(b.z, b.w);
  }
  return r;
}

// What lifted entries carry (see qskinny.hip).
template <int FMT>
__device__ __forceinline__ float q_lift(const QLayer& L) {
  return FMT == QF_E8 ? 68.f : 128.f + (float)(L.K / 2);
}
// Uniform levels by arithmetic alone, in units of their step: in bfloat16 lifted,
// 128 + q is 0x4300 | q; in float16, whose 1024 + q is 0x6400 | q and which adds
// in pairs, the entry itself, code - K / 2.
template <int FMT, typename T>
__device__ __forceinline__ v4u q_decode_lifted(const QLayer& L, const uint4& c, int s) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  v4u r;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    uint32_t q;
    if constexpr (FMT == QF_NIB) q = (w[s] >> (4 * b)) & 0x000f000fu;
    else q = (w[2 * s + (b >> 1)] >> (8 * (b & 1))) & 0x00ff00ffu;
    if constexpr (T::HALF) {
      const v2h mid = {(_Float16)(float)(-1024 - L.K / 2), (_Float16)(float)(-1024 - L.K / 2)};
      r[b] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, q | 0x64006400u) + mid);
    } else {
      r[b] = q | 0x43004300u;
    }
  }
  return r;
}

// ------------------------------------------------------------------ epilogue

enum QAct : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

__device__ __forceinline__ float act_fwd(int act, float u) {
  switch (act) {
    case ACT_RELU: return u < 0.f ? 0.f : u;   // keeps NaN
    case ACT_GELU: return 0.5f * u * (1.f + erff(u * 0.70710678f));
    case ACT_GELU_TANH: return 0.5f * u * (1.f + tanhf(0.79788456f * (u + 0.044715f * u * u * u)));
    case ACT_SILU: return u / (1.f + expf(-u));
  }
  return u;
}
__device__ __forceinline__ float act_slope(int act, float u) {
  switch (act) {
    case ACT_RELU: return u > 0.f ? 1.f : u == u ? 0.f : u;
    case ACT_GELU: {
      // (a u beyond float16 is kept as an infinity: u times the density is 0 there, not inf * 0)
      const float d = expf(-0.5f * u * u);
      return 0.5f * (1.f + erff(u * 0.70710678f)) + (d == 0.f ? 0.f : u * 0.39894228f * d);
    }
    case ACT_GELU_TANH: {
      const float th = tanhf(0.79788456f * (u + 0.044715f * u * u * u));
      // 1 - th^2 is 0 where u^3 overflows; the product must not be inf * 0
      const float q = 1.f - th * th;
      return 0.5f * (1.f + th) + (q == 0.f ? 0.f : 0.5f * u * q * 0.79788456f * (1.f + 0.134145f * u * u));
    }
    case ACT_SILU: {
      const float q = 1.f / (1.f + expf(-u));
      return q == 0.f || q == 1.f ? q : q * (1.f + u * (1.f - q));   // (its ends: not inf * 0)
    }
  }
  return 1.f;
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == DT_F32) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == DT_BF16 ? OpBf16::val(b) : OpF16::val(b);
}

// Four consecutive elements at p[i], as many as `live`; vec: 4-element aligned.
__device__ __forceinline__ void load4(const void* p, int64_t i, int dtype, bool vec, int live, float* v) {
  if (vec && live >= 4) {
    if (dtype == DT_F32) {
      const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t h[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = dtype == DT_BF16 ? OpBf16::val(h[k]) : OpF16::val(h[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < live ? load_as_f32(p, i + k, dtype) : 0.f;
  }
}
__device__ __forceinline__ void store4(void* p, int64_t i, int dtype, bool vec, int live, const float* v) {
  if (vec && live >= 4) {
    if (dtype == DT_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else if (dtype == DT_BF16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          make_uint2(OpBf16::pack(v[0], v[1]), OpBf16::pack(v[2], v[3]));
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          make_uint2(OpF16::pack(v[0], v[1]), OpF16::pack(v[2], v[3]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= live) break;
      if (dtype == DT_F32)
        static_cast<float*>(p)[i + k] = v[k];
      else
        static_cast<uint16_t*>(p)[i + k] = (uint16_t)(dtype == DT_BF16 ? OpBf16::bits(v[k]) : OpF16::bits(v[k]));
    }
  }
}
#endif  // __HIPCC__

// Operands of the float16 products carry a power of two per row that takes the
// row's largest magnitude to [2^14, 2^15): float16's eleven bits then hold
// elements down to 2^-28 of it in full and smaller ones to 2^-39 of it, below
// what float32 sums resolve.  The factor comes from the bits of that magnitude;
// a row of zeros, or one that holds NaN or infinities, keeps factor 1.
#ifdef __HIPCC__
__device__ __forceinline__ int pow2_shift(uint32_t maxbits) {
  const int e = (int)(maxbits >> 23) & 255;
  return maxbits == 0 || e == 255 ? 0 : min(141 - max(e, 1), 126);
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }   // |k| <= 126
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// x in two float16 terms.
__device__ __forceinline__ void f16_terms(float x, uint32_t* b) {
  b[0] = OpF16::bits(x);
  const float lo = x - OpF16::val(b[0]);
  b[1] = fabsf(x) <= 65504.f ? OpF16::bits(lo) : 0u;   // an infinite or NaN x stays what it is, alone
}
#endif

// The outputs of a product, out[j][i] for row j and column i: four consecutive
// columns at a time.
struct QOut {
  void* y; int64_t ldy;
  void* pre; int64_t ldpre;         // the activation's argument (nullptr: not kept)
  const void* res; int64_t ldres;   // added after the activation
  const float* bias;                // per column
  const uint32_t* rowmax;           // per row: its operand's largest magnitude (pow2_shift; nullptr: no factor)
  const uint32_t* colmax;           // per column, likewise
  const float* colscale;            // per column: factor of the product (nullptr: 1)
  const float* coloff;              // per column: factor of rowadd
  const float* rowadd;              // per row: added, times coloff + colscale mid if there is a colscale
  const float* levels; int mid;     // d = 1: levels[mid] (mid < 0: zero)
  int act, dtype;
  int vec;                          // 4-element alignment of y, pre, res
  int64_t rows, cols;
};

#ifdef __HIPCC__
// What four columns multiply and add: u = a v + o rowadd + b.
struct QCol {
  float a[4], o[4], b[4];
  int live;   // columns there are (<= 0: none)
};
// (vectors of the columns may begin at any element)
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ QCol q_col4(const QOut& O, int64_t i) {
  QCol C;
  C.live = (int)min((int64_t)4, O.cols - i);
  const float mid = O.colscale && O.mid >= 0 ? O.levels[O.mid] : 0.f;
  v4f_any b = {0.f, 0.f, 0.f, 0.f}, a = {1.f, 1.f, 1.f, 1.f}, o = b;
  v4u_any top = {0u, 0u, 0u, 0u};   // (factor 1)
  if (C.live == 4) {   // all of them on their way together
    if (O.bias) b = *reinterpret_cast<const v4f_any*>(O.bias + i);
    if (O.colscale) a = *reinterpret_cast<const v4f_any*>(O.colscale + i);
    if (O.colscale && O.coloff) o = *reinterpret_cast<const v4f_any*>(O.coloff + i);
    if (O.colmax) top = *reinterpret_cast<const v4u_any*>(O.colmax + i);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (k >= C.live) continue;
      if (O.bias) b[k] = O.bias[i + k];
      if (O.colscale) a[k] = O.colscale[i + k];
      if (O.colscale && O.coloff) o[k] = O.coloff[i + k];
      if (O.colmax) top[k] = O.colmax[i + k];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    C.b[k] = b[k];
    C.a[k] = a[k];
    C.o[k] = O.colscale ? fmaf(a[k], mid, o[k]) : 1.f;
    C.a[k] *= pow2(-pow2_shift(top[k]));
  }
  return C;
}
// Row j's part of it.
__device__ __forceinline__ void q_affine4(const QOut& O, const QCol& C, int64_t j, float* v) {
  const float f = O.rowmax ? pow2(-pow2_shift(O.rowmax[j])) : 1.f;
  const float add = O.rowadd ? O.rowadd[j] : 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = fmaf(C.a[k], v[k] * f, (O.rowadd ? C.o[k] * add : 0.f) + C.b[k]);
}

// Four columns of row j: y = act(affine of v + bias) + res.
__device__ __forceinline__ void q_finish4(const QOut& O, int64_t j, int64_t i, float* v) {
  const QCol C = q_col4(O, i);
  if (j >= O.rows || C.live <= 0) return;
  q_affine4(O, C, j, v);
  if (O.pre) store4(O.pre, j * O.ldpre + i, O.dtype, O.vec, C.live, v);
  if (O.act != ACT_NONE)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = act_fwd(O.act, v[k]);
  if (O.res) {
    float r[4];
    load4(O.res, j * O.ldres + i, O.dtype, O.vec, C.live, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += r[k];
  }
  store4(O.y, j * O.ldy + i, O.dtype, O.vec, C.live, v);
}

// The entries of row i's columns j .. j + 3 (j a multiple of 4, inside the packed
// chunks): the code's bits first, then the entries, so that loads of several
// quads can be on their way together.
// (A row's code lies 16 bytes after the one before it, within their sixteen: q_code4_at for
// the sixteen's first, q_code4_of for a row of them.)
__device__ __forceinline__ const uint16_t* q_code4_at(const QLayer& L, int64_t block, int64_t j) {
  const int steps = q_steps(L.fmt);
  const int64_t blk = j >> 3, c = blk / (4 * steps);
  const int kb = (int)(blk & 3), s = (int)(blk - c * 4 * steps) >> 2, half = (int)(j >> 2) & 1;
  const size_t at = (((size_t)block * L.chunks + c) * 64 + kb * 16) * 8;   // 16-bit words
  return reinterpret_cast<const uint16_t*>(L.packed) + at + (L.fmt == QF_NIB ? s * 2 : L.fmt == QF_BYTE ? s * 4 + half * 2 : s);
}
__device__ __forceinline__ uint32_t q_code4_of(const QLayer& L, const uint16_t* first, int row) {
  first += row * 8;
  return L.fmt == QF_NIB || L.fmt == QF_BYTE ? *reinterpret_cast<const uint32_t*>(first) : *first;
}
__device__ __forceinline__ uint32_t q_code4(const QLayer& L, int64_t i, int64_t j) {
  return q_code4_of(L, q_code4_at(L, i >> 4, j), (int)(i & 15));
}
// (base, step: of uniform levels)
struct QLevels {
  float base, step;
};
__device__ __forceinline__ QLevels q_levels(const QLayer& L) {
  QLevels v = {0.f, 0.f};
  if ((L.fmt == QF_NIB || L.fmt == QF_BYTE) && L.uniform) {
    v.base = L.levels[0];
    v.step = L.levels[1] - v.base;
  }
  return v;
}
__device__ __forceinline__ void q_entries4(const QLayer& L, const QLevels& v, uint32_t code, int64_t j, float* e) {
  const int half = (int)(j >> 2) & 1;
  if (L.fmt == QF_NIB || L.fmt == QF_BYTE) {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      q[k] = L.fmt == QF_NIB ? (code >> (8 * half + 4 * (k >> 1) + 16 * (k & 1))) & 15u
                             : (code >> (8 * (k >> 1) + 16 * (k & 1))) & 63u;
    if (L.uniform) {   // (exactly the same, and no look-up)
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = fmaf((float)q[k], v.step, v.base);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = L.levels[q[k]];
    }
  } else if (L.fmt == QF_E8) {
    const uint32_t w = q_e8_nibbles(L, L.lut, code);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      e[k] = 0.5f * (float)((int)((w >> (8 * half + 4 * (k >> 1) + 16 * (k & 1))) & 15u) - 8);
  } else {
    const float4 q = *reinterpret_cast<const float4*>(L.e32 + (size_t)code * 8 + half * 4);
    e[0] = q.x; e[1] = q.y; e[2] = q.z; e[3] = q.w;
  }
}
__device__ __forceinline__ void q_entries4(const QLayer& L, uint32_t code, int64_t j, float* e) {
  q_entries4(L, q_levels(L), code, j, e);
}
#endif

// ------------------------------------------------------------------ launchers

// D[j][i] = sum over the plane pairs (p, q) and k of A_p[i][k] B_q[j][k] (16-bit
// planes, K a multiple of 32; B may stay in rows of ldb elements, a multiple of 8,
// 16-byte aligned), then
// O, or the contraction.  part (split K): splits x rows x cols float32.
// Operand order of a plane: sixteen rows by 32 columns after another, along the
// row first, each a contiguous KB of its rows (64 bytes each).  K: the plane's
// columns, a multiple of 32; its rows are padded to a multiple of 16.
__device__ __forceinline__ int64_t q_at(int64_t row, int64_t k, int64_t K) {
  return ((row >> 4) * (K >> 5) + (k >> 5)) * 512 + (row & 15) * 32 + (k & 31);
}
struct QGemm {
  const uint16_t* A; int64_t lda, planeA;   // operand order (lda = 0), or rows, as B's
  int64_t acols, arows;                     // of an A that lies transposed (qgemm_tile.h)
  const uint16_t* B; int64_t ldb, planeB;   // operand order (ldb = 0), or rows
  int64_t M, N, K;        // columns i, rows j, depth of one plane
  int npairs;
  uint8_t pa[4], pb[4];
  bool bf16;              // bfloat16 operands (else float16)
  QOut O;
  // Contraction (cpart != nullptr), D the gradient of layer rows row0 + j: per
  // 64 columns the sums of e D and of D, cpart[split][j][block] (float2), in
  // place of an output.
  QLayer L;
  int64_t row0;
  float2* cpart; int64_t cblocks;
};
constexpr int Q_CONTRACT = 64;
// Pairs of PA and PB planes whose orders add to at most one.
void q_pairs(QGemm& g, int PA, int PB);
int q_gemm_splits(int64_t M, int64_t N, int64_t K, int npairs);
size_t q_gemm_workspace(int64_t M, int64_t N, int64_t K, int npairs);
hipError_t launch_q_gemm(const QGemm& g, float* part, hipStream_t st);

// The product with few rows (qskinny.hip): x in place (16-bit rows of ldx > 0
// elements, 16-byte aligned, n a multiple of 8), or in operand order (ldx = 0):
// planes of whole chunks, 16 rows by 16 rows, each step's 64 lanes x 16 bytes
// together.  Two planes: float16, with O.rowmax (one float16 plane: with or without).  Column groups need chunks that
// lie in one group.
bool q_skinny_ok(const QLayer& L);
bool q_few_rows(const QLayer& L, int dtype, int64_t t);   // whether a product of t rows should take it (qlinear.hip)
hipError_t launch_q_skinny(const QLayer& L, const uint16_t* x, int64_t ldx, int64_t planex, int64_t t, int planes,
                           bool bf16, const QOut& O, hipStream_t st);

struct QLinearArgs {
  QLayer L;
  const void* x; int64_t ldx;
  int dtype;
  int64_t t;
  const float* bias;
  int act;
  const void* res; int64_t ldres;
  void* y; int64_t ldy;
  void* pre; int64_t ldpre;
};
struct QLinearGrad {
  QLayer L;
  const void* dy; int64_t lddy;
  const void* x; int64_t ldx;
  const void* pre; int64_t ldpre;
  int dtype, act;
  int64_t t;
  bool need_dx, need_dlayer;
  void* dx; int64_t lddx;
  float *dscale, *doffset, *dbias;
};
// A layer from a C entry's arguments, checked (api_ops.hip): its shapes and format, and
// with its pointers.
int q_layer_shape(QLayer& L, int64_t m, int64_t n, int64_t K, int64_t d, int64_t group, int kind);
int q_layer_of(QLayer& L, const void* packed, int64_t m, int64_t n, const mpq_codebook* cb, const float* scale,
               const float* offset, int64_t group);

size_t q_packed_bytes(const QLayer& L);
hipError_t launch_q_pack(const int32_t* codes, const QLayer& L, void* packed, hipStream_t st);
size_t q_linear_workspace(const QLinearArgs& A);
hipError_t launch_q_linear(const QLinearArgs& A, void* ws, hipStream_t st);
size_t q_grad_workspace(const QLinearGrad& A);
hipError_t launch_q_grad(const QLinearGrad& A, void* ws, hipStream_t st);
// Parts of them, float16: a layer's planes in operand order (planes = 0: entries; else
// terms of its weights times 2^pow2_shift(refs)), the bounds refs, and the affine's sums
// of a dW that is contracted (cpart) or in memory.
hipError_t launch_q_unpack(const QLayer& L, int64_t Kp, int planes, const uint32_t* refs, uint16_t* out, int64_t plane,
                           hipStream_t st);
hipError_t launch_q_bounds(const QLayer& L, uint32_t* refs, hipStream_t st);
hipError_t launch_q_affine_sums(const QLayer& L, const float2* cpart, int splits, int64_t cblocks, const float* dW, int64_t ldw,
                                float* dscale, float* doffset, hipStream_t st);
hipError_t launch_q_zero_rows(void* p, int64_t rows, int64_t cols, int64_t ld, int dtype, hipStream_t st);

// What mpq_codebook_prepare notes in the low bits of mpq_codebook.magic (the struct
// keeps the size that callers were built with): whether packed layers can hold the
// entries (d = 1: their differences to level K / 2), exact in bfloat16 and in
// float16, and whether (d = 1) the levels are evenly spaced, too.
constexpr uint64_t CB_NARROW = 1, CB_EVEN = 2, CB_NOTES = CB_NARROW | CB_EVEN;

// Host images of an E8 prefix's decoder table and code map (K each at most);
// false if the codebook does not have the shells' structure.
bool q_e8_tables(const float* cb, int64_t K, uint32_t* lut, uint16_t* map, int* entries, int* pairs);
int64_t q_e8_shell(int h);
int q_e8_pairs(int64_t K);   // table entries that stand for a point and its negative

}  // namespace mpq
