// The product of a solved layer with few rows, straight from its packed codes.
//
// Mathematics.  z[i] = sum_j e_ij x_j with the codebook's entries as they are
// (exact in 16 bits) and float32 sums, then u = a z + o' sum_j x_j: no weight is
// ever formed, so none is rounded.  The sum over x rides along as one more
// matrix product, with a row of ones in the layer's place.  float32 x enters as
// two float16 terms (22 bits) of x times a power of two per token.
// With bfloat16 x, E8's entries and evenly spaced levels enter lifted: 64 + q / 2
// and 128 + q are the code's bits under a constant exponent, two instructions a
// pair where the entry itself takes six.  The lift comes off again unit by unit
// (128 columns), with the sum over x, before its part could outgrow float32's
// bits (a unit's sum is rounded at 2^-24 of some 140 sum |x|: far under half a
// bfloat16 step of the result).
//
// Bound.  HBM traffic is the packed codes (2 bits a weight for E8); what the
// waves wait on is their own decoding (some 20 instructions a step of 64 blocks
// for E8 and its table's look-ups) and, from two token tiles on, the operand
// loads.  A wave's matrix operand is what its lanes decode, sixteen rows at a
// time, so the sixteen columns of the other operand are tokens: one token costs
// what sixteen do but for x's loads.
//
// Split.  A workgroup takes R tiles of 16 rows, its waves the chunks of the tiles
// in turn, and joins their sums in a fixed order through LDS.  E8's table (148 KB
// for 65536 points) fills a CU's LDS, so those workgroups stay, one per CU, and
// take tile after tile.  x lies in operand order (1 KB a load, whole lines): in
// place its sixteen rows often start a multiple of 4 KB apart, on the same few
// cache channels, 64 clocks a load instead of 16.
//
// Measured (microseconds at 1, 16, 32, 64, 128 tokens, bfloat16, one layer again
// and again, so that its codes come from the last-level cache): E8 4096 x 14336
// 12.1, 16.0, 21.0, 31.5, 56; 4096 x 4096 8.0, 10.1, 12.9, 15.5, 26; 32768 x 4096
// 23, 28, 46, 67, 124; four bits 4096 x 14336 7.9, 12.4, 18.1, 28, 48; 32768 x 4096
// 15.6, 23, 41, 61, 113.  An empty call (64 columns) is 6.3 with E8's table and 3.9
// without.  One token through layers in turn, whose codes come from HBM (more than
// 256 MB of them), against one layer again: E8 4096 x 14336 13.4 | 12.6, 32768 x
// 4096 24.2 | 24.1; four bits 12.2 | 8.5, 19.3 (3.5 TB/s of codes) | 17.3.
#include <algorithm>
#include <type_traits>
#include "qlayer.h"

namespace mpq {

namespace {

// Sixteen waves where a wave's operands fit 128 registers, else eight (one token,
// 4096 x 14336: eight waves 16 us for E8 and 11 for four bits, sixteen 14 and 10,
// before the loads were counted).
constexpr int sk_waves(int XP, int NT, int R, bool grouped) { return XP * NT * R == 1 && !grouped ? 16 : 8; }

// Whether entries are looked up: all but evenly spaced levels and those of the
// generic codebook, which come straight from memory.
constexpr bool sk_table(int f, bool uni) { return f == QF_E8 || (f != QF_VEC && !uni); }

struct SkinnyArgs {
  QLayer L;
  const uint16_t* x; int64_t ldx, planex;   // ldx = 0: operand order
  int kblocks;          // blocks of eight columns that x holds
  uint32_t xbytes;      // of one plane
  int64_t t;
  bool has_offset;
  int lut_words;
  uint32_t ginv;        // 2^32 over a group's units, rounded up; 0: one unit
  QOut O;
};

// What a wave takes at a time: four steps (half a chunk of d = 8 codes), or a
// whole chunk of two.
constexpr int unit_steps(int f) { return q_steps(f) < 4 ? q_steps(f) : 4; }

// 16 or 8 bytes at p[at], zeros from `bytes` on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
__device__ __forceinline__ v4u load_words(const void* p, uint32_t bytes, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b128(buffer_of(p, bytes), at, 0, 0);
}
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v2u load_half(const void* p, uint32_t bytes, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b64(buffer_of(p, bytes), at, 0, 0);
}
template <int N>
__device__ __forceinline__ uint4 load_buffer(const void* p, uint32_t bytes, uint32_t at) {
  if constexpr (N == 16) {
    const v4u w = load_words(p, bytes, at);
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const v2u w = load_half(p, bytes, at);
    return make_uint4(w[0], w[1], 0, 0);
  }
}
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED, bool UNI>
__global__ __launch_bounds__(64 * sk_waves(XP, NT, R, GROUPED)) void q_skinny_kernel(SkinnyArgs A) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int US = unit_steps(FMT), UPC = q_steps(FMT) / US;
  constexpr int SUBS = R * NT, SK_WAVES = sk_waves(XP, NT, R, GROUPED);
  constexpr bool TABLE = sk_table(FMT, UNI);
  static_assert(SUBS <= SK_WAVES, "a wave adds up one subtile");
  // one subtile's worth of sums beside the table, or all of them over it once
  // no more tile needs it (E8), or beside it (the others' tables are small)
  constexpr bool OVER = FMT == QF_E8;
  uint32_t* lut = lds;
  v4f* red = reinterpret_cast<v4f*>(lds + (TABLE ? A.lut_words : 0));
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, kb = lane >> 4;
  const int64_t tok0 = (int64_t)blockIdx.y * (16 * NT);
  const int tgs = (A.L.tiles + R - 1) / R, units = A.L.chunks * UPC;
  // tokens past the last repeat it: a token's sums are its own column's
  uint32_t xrow[NT];   // in bytes
  const int xstep = A.ldx ? 64 : 1024;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xrow[n] = A.ldx ? (uint32_t)(min(tok0 + n * 16 + r, A.t - 1) * A.ldx * 2) + kb * 16
                    : (uint32_t)(min(tok0 / 16 + n, (A.t - 1) / 16) * (units * US)) * 1024u + lane * 16;

  struct Codes {
    uint4 v[R];
    float scale[R][4], offset[R][4];   // GROUPED: of the unit's group
  };
  struct Xs {
    v4u v[US][NT][XP];
  };
  // No load stands under a branch (past the last unit and past x's columns the
  // buffers' bounds give zeros): what a use waits for is then a constant number of
  // loads back, and the ones after it stay on their way.
  auto load_codes = [&](Codes& c, int tg, int u) {
#pragma unroll
    for (int q = 0; q < R; ++q) {   // a tile past the last repeats it; its sums are not stored
      const int tile = min(tg * R + q, A.L.tiles - 1);
      const uint4* p = A.L.packed + (size_t)tile * A.L.chunks * 64;
      const uint32_t bytes = (uint32_t)A.L.chunks * 1024, at = (uint32_t)(u / UPC * 64 + lane) * 16 + u % UPC * 8;
      c.v[q] = load_buffer<UPC == 1 ? 16 : 8>(p, bytes, at);
      if constexpr (GROUPED) {
        // the unit (a chunk) lies in one group
        const uint32_t in = (uint32_t)min(u, units - 1);
        const int64_t g = A.ginv ? __umulhi(in, A.ginv) : in;
        const float* off = A.L.offset ? A.L.offset : A.L.scale;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t i = min((int64_t)tile * 16 + 4 * kb + v, A.L.m - 1) * A.L.G + g;
          c.scale[q][v] = A.L.scale[i];
          c.offset[q][v] = off[i];
        }
      }
    }
  };
  auto load_x = [&](Xs& x, int u) {
#pragma unroll
    for (int s = 0; s < US; ++s) {
      const bool in = (u * US + s) * 4 + kb < A.kblocks;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < XP; ++p)
          x.v[s][n][p] = load_words(A.x + p * A.planex, A.xbytes, in ? xrow[n] + (uint32_t)((u * US + s) * xstep) : A.xbytes);
    }
  };
  // A unit's codes are loaded two units ahead, its x two or, where the registers
  // are wanted, one.
  constexpr int XD = NT * XP <= 2 ? 2 : 1;
  Codes next[2];
  Xs xnext[XD];
  auto load_first = [&](int tg, int first) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // (in the order of their uses)
      load_codes(next[h], tg, first + h * SK_WAVES);
      if (h < XD) load_x(xnext[h], first + h * SK_WAVES);
      keep_order();
    }
  };
  if (TABLE) {
    q_lut_fill<FMT, T>(A.L, lut, 64 * SK_WAVES);
    keep_order();
  }
  load_first(blockIdx.x, wave);
  if (TABLE) {
    if (FMT == QF_E8) q_lut_wait<2 * R + XD * US * NT * XP>();
    __syncthreads();
  }
  const float mid = q_centre(A.L), step = UNI && FMT != QF_E8 ? A.L.levels[1] - A.L.levels[0] : 1.f;
  constexpr bool LIFTED = UNI && !T::HALF;   // decoded entries carry q_lift
  const float lift = LIFTED ? q_lift<FMT>(A.L) : 0.f;
  for (int tg = blockIdx.x; tg < tgs; tg += gridDim.x) {
    const bool more = FMT == QF_E8 && tg + (int)gridDim.x < tgs;   // (the others' grids have a workgroup per tile)
    // this wave's part of the epilogue's operands, and the affine, early
    const int64_t tok = tok0 + wave % NT * 16 + r, i0 = (int64_t)(tg * R + wave / NT) * 16 + 4 * kb;
    float res[4] = {0.f, 0.f, 0.f, 0.f}, bias[4] = {0.f, 0.f, 0.f, 0.f};
    const int live = wave < SUBS && tok < A.t ? (int)min((int64_t)4, A.O.cols - i0) : 0;
    if (live > 0) {
      if (A.O.res) load4(A.O.res, tok * A.O.ldres + i0, A.O.dtype, A.O.vec, live, res);
      if (A.O.bias)
#pragma unroll
        for (int k = 0; k < 4; ++k) bias[k] = k < live ? A.O.bias[i0 + k] : 0.f;
    }
    float sa[R][4], so[R][4];
    if (!GROUPED)
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t i = min((int64_t)(tg * R + q) * 16 + 4 * kb + v, A.L.m - 1);
          sa[q][v] = A.L.scale[i];
          so[q][v] = A.has_offset && A.L.offset ? A.L.offset[i] : 0.f;
        }
    v4f acc[R][NT], xs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xs[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < R; ++q) acc[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    auto unit = [&](Codes& code, Xs& x, int u, auto reload) {
      // the table's words of the whole unit first: one wait for LDS, not one a step
      uint32_t nib[R][US];
      if constexpr (FMT == QF_E8)
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int s = 0; s < US; ++s)
            nib[q][s] = q_e8_nibbles(A.L, lut, (s < 2 ? code.v[q].x : code.v[q].y) >> (16 * (s & 1)));
      keep_order();
      constexpr bool FRESH = GROUPED || LIFTED;   // this unit's sum over x apart
      v4f z[R][NT], zx[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (FRESH) zx[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (GROUPED) z[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int s = 0; s < US; ++s) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          v4u w;
          if constexpr (FMT == QF_E8) w = UNI ? q_e8_lifted(nib[q][s]) : q_e8_entries<T>(nib[q][s]);
          else if constexpr (UNI) w = q_decode_lifted<FMT, T>(A.L, code.v[q], s);
          else w = q_decode<FMT, T>(A.L, lut, code.v[q], s);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              if (GROUPED) z[q][n] = T::mfma(w, x.v[s][n][p], z[q][n]);
              else acc[q][n] = T::mfma(w, x.v[s][n][p], acc[q][n]);
            }
        }
        if (LIFTED || A.has_offset) {
          const v4u one = {T::ONES, T::ONES, T::ONES, T::ONES};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              if (FRESH) zx[n] = T::mfma(one, x.v[s][n][p], zx[n]);
              else xs[n] = T::mfma(one, x.v[s][n][p], xs[n]);
            }
        }
      }
      if (LIFTED)
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            v4f& c = GROUPED ? z[q][n] : acc[q][n];
#pragma unroll
            for (int v = 0; v < 4; ++v) c[v] = fmaf(-lift, zx[n][v], c[v]);
          }
      if (GROUPED) {
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float a = code.scale[q][v], o = fmaf(a, mid, A.L.offset ? code.offset[q][v] : 0.f);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[q][n][v] = fmaf(a * step, z[q][n][v], fmaf(o, zx[n][v], acc[q][n][v]));
          }
      } else if (LIFTED && A.has_offset) {
#pragma unroll
        for (int n = 0; n < NT; ++n) xs[n] += zx[n];
      }
      if (reload.value) {
        load_codes(code, tg, u + 2 * SK_WAVES);
        load_x(x, u + XD * SK_WAVES);
        keep_order();
      }
    };
    // (one way round the loop, so that every turn finds the same loads behind it)
    int u = wave;
    for (; u + SK_WAVES < units; u += 2 * SK_WAVES) {
      unit(next[0], xnext[0], u, std::true_type{});
      unit(next[1], xnext[XD - 1], u + SK_WAVES, std::true_type{});
    }
    if (u < units) unit(next[0], xnext[0], u, std::false_type{});
    // (not under a branch either; after the last tile nothing)
    if constexpr (FMT == QF_E8) load_first(more ? tg + gridDim.x : tg, more ? wave : units);
    if (!GROUPED) {
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float o = A.has_offset ? fmaf(sa[q][v], mid, so[q][v]) : 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[q][n][v] = fmaf(sa[q][v] * step, acc[q][n][v], A.has_offset ? o * xs[n][v] : 0.f);
        }
    }
    // Subtile (q, n) is added up, in the order of the waves, by wave (q NT + n).
    float mine[4] = {0.f, 0.f, 0.f, 0.f};
    if (OVER && more) {
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int dst = q * NT + n;
          if (wave != dst) red[(wave < dst ? wave : wave - 1) * 64 + lane] = acc[q][n];
          __syncthreads();
          if (wave == dst)
            for (int w = 0; w < SK_WAVES; ++w) {
              const v4f p = w == dst ? acc[q][n] : red[(w < dst ? w : w - 1) * 64 + lane];
#pragma unroll
              for (int k = 0; k < 4; ++k) mine[k] += p[k];
            }
          __syncthreads();
        }
    } else {
      v4f* all = OVER ? reinterpret_cast<v4f*>(lds) : red;
      if (OVER) __syncthreads();   // every wave is done with the table
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) all[((q * NT + n) * SK_WAVES + wave) * 64 + lane] = acc[q][n];
      __syncthreads();
      if (wave < SUBS)
#pragma unroll
        for (int w = 0; w < SK_WAVES; ++w) {
          const v4f p = all[(wave * SK_WAVES + w) * 64 + lane];
#pragma unroll
          for (int k = 0; k < 4; ++k) mine[k] += p[k];
        }
      if (more) __syncthreads();
    }
    if (live > 0) {
      if (A.O.rowmax) {
        const float f = pow2(-pow2_shift(A.O.rowmax[tok]));
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[k] *= f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mine[k] += bias[k];
      if (A.O.pre) store4(A.O.pre, tok * A.O.ldpre + i0, A.O.dtype, A.O.vec, live, mine);
      if (A.O.act != ACT_NONE)
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[k] = act_fwd(A.O.act, mine[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) mine[k] += res[k];
      store4(A.O.y, tok * A.O.ldy + i0, A.O.dtype, A.O.vec, live, mine);
    }
    if (FMT != QF_E8) break;
  }
}

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED, bool UNI>
hipError_t launch(const SkinnyArgs& A, hipStream_t st) {
  constexpr int SK_WAVES = sk_waves(XP, NT, R, GROUPED);
  const int tgs = (A.L.tiles + R - 1) / R;
  const int wgs = FMT == QF_E8 ? std::min(tgs, 256) : tgs;
  const size_t table = sk_table(FMT, UNI) ? (size_t)A.lut_words * 4 : 0, tile = 64 * sizeof(v4f);
  const size_t shared = FMT == QF_E8 ? std::max(table + (SK_WAVES - 1) * tile, R * NT * SK_WAVES * tile)
                                     : table + R * NT * SK_WAVES * tile;
  hipLaunchKernelGGL((q_skinny_kernel<FMT, T, XP, NT, R, GROUPED, UNI>),
                     dim3((unsigned)wgs, (unsigned)((A.t + 16 * NT - 1) / (16 * NT))), dim3(64 * SK_WAVES), shared, st, A);
  return hipGetLastError();
}

template <int FMT, typename T, int XP, int NT, bool GROUPED, bool UNI>
hipError_t pick_rows(const SkinnyArgs& A, hipStream_t st) {
  // two tiles per workgroup share x's loads, once that still leaves every CU one
  if constexpr (XP == 1 && NT * (GROUPED ? 2 : 1) <= 2 && (FMT == QF_E8 || FMT == QF_NIB))
    if (A.L.tiles >= 512) return launch<FMT, T, XP, NT, 2, GROUPED, UNI>(A, st);
  return launch<FMT, T, XP, NT, 1, GROUPED, UNI>(A, st);
}

template <int FMT, typename T, int XP, bool GROUPED, bool UNI>
hipError_t pick_tokens(const SkinnyArgs& A, hipStream_t st) {
  if (A.t <= 16) return pick_rows<FMT, T, XP, 1, GROUPED, UNI>(A, st);
  // Four tiles of 16 tokens share a decoding, or five where that saves a round of
  // workgroups, one on each of the 256 CUs.
  // Measured, five | four, bfloat16: 80 tokens of 2304 x 8192 E8 24.8 | 33.3 us,
  // four bits 21.3 | 28.1, 8 bits 21.7 | 27.8, generic 31 | 47; of 2048 x 8192 (256
  // workgroups of four) 24.7 | 21.6, 21.3 | 19.0, 21.7 | 19.2, 31 | 31; 160 tokens of
  // four bits 4096 x 4096 24.9 | 28.0; 1024 x 1024 E8, 160 tokens 11.3 | 10.5, 320
  // 12.4 | 16.4, 384 (two rounds either way) 18.2 | 16.5; float16 alike.
  if constexpr (XP == 1) {
    const int64_t tgs = A.L.tiles;
    if ((tgs * ((A.t + 79) / 80) + 255) / 256 < (tgs * ((A.t + 63) / 64) + 255) / 256)
      return pick_rows<FMT, T, XP, 5, GROUPED, UNI>(A, st);
    if (A.t > 32) return pick_rows<FMT, T, XP, 4, GROUPED, UNI>(A, st);
  }
  return pick_rows<FMT, T, XP, 2, GROUPED, UNI>(A, st);
}

template <int FMT, typename T, int XP, bool GROUPED>
hipError_t pick_levels(const SkinnyArgs& A, hipStream_t st) {
  // (float32 x keeps the table: the lifted sums would cost it bits)
  if constexpr (XP == 1)
    if (A.L.uniform) return pick_tokens<FMT, T, XP, GROUPED, true>(A, st);
  return pick_tokens<FMT, T, XP, GROUPED, false>(A, st);
}

template <typename T, int XP>
hipError_t pick_format(const SkinnyArgs& A, hipStream_t st) {
  const bool grouped = A.L.G > 1;
  switch (A.L.fmt) {
    case QF_NIB: return grouped ? pick_levels<QF_NIB, T, XP, true>(A, st) : pick_levels<QF_NIB, T, XP, false>(A, st);
    case QF_BYTE: return grouped ? pick_levels<QF_BYTE, T, XP, true>(A, st) : pick_levels<QF_BYTE, T, XP, false>(A, st);
    case QF_E8: return pick_tokens<QF_E8, T, XP, false, !T::HALF>(A, st);
    default: return pick_tokens<QF_VEC, T, XP, false, false>(A, st);
  }
}

}  // namespace

bool q_skinny_ok(const QLayer& L) { return L.G == 1 || L.group % q_chunk(L.fmt) == 0; }

hipError_t launch_q_skinny(const QLayer& L, const uint16_t* x, int64_t ldx, int64_t planex, int64_t t, int planes,
                           bool bf16, const QOut& O, hipStream_t st) {
  SkinnyArgs A;
  A.L = L;
  A.x = x;
  A.ldx = ldx;
  A.planex = planex;
  A.kblocks = (int)(ldx ? L.n / 8 : (int64_t)L.chunks * q_chunk(L.fmt) / 8);
  A.xbytes = (uint32_t)(ldx ? ((t - 1) * ldx + L.n) * 2 : (t + 15) / 16 * 16 * A.kblocks * 16);
  A.t = t;
  A.has_offset = L.has_offset();
  A.lut_words = (q_lut_words(L.fmt, L.lut_entries) + 3) / 4 * 4;
  A.O = O;
  const uint64_t per = L.G > 1 ? (uint64_t)(L.group / q_chunk(L.fmt)) : 1;
  A.ginv = per > 1 ? (uint32_t)(((1ull << 32) + per - 1) / per) : 0;   // (units and per are below 2^16: exact)
  if (bf16) return pick_format<OpBf16, 1>(A, st);
  return planes == 2 ? pick_format<OpF16, 2>(A, st) : pick_format<OpF16, 1>(A, st);
}

}  // namespace mpq
