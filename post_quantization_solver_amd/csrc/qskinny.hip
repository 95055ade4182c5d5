// The product of a solved layer with few rows, straight from its packed codes.
//
// Mathematics.  z[i] = sum_j e_ij x_j with the codebook's entries as they are
// (exact in 16 bits) and float32 sums, then u = a z + o' sum_j x_j: no weight is
// ever formed, so none is rounded.  The sum over x rides along as one more
// matrix product, with a row of ones in the layer's place.  float32 x enters as
// two float16 terms (22 bits) of x times a power of two per token.
// Evenly spaced levels need no table: 128 + code is the code's bits under a
// constant exponent in bfloat16.  The 128 and the middle level come off again
// unit by unit (128 columns), with the sum over x, before their part could
// outgrow float32's bits (a unit's sum is rounded at 2^-24 of some 140 sum |x|:
// far under half a bfloat16 step of the result).
//
// Bound.  HBM traffic is the packed codes (2 bits a weight for E8); what the
// waves wait on is their own decoding (some 30 instructions a step of 64 blocks)
// and, from two token tiles on, the operand loads.  A wave's matrix operand is
// what its lanes decode, sixteen rows at a time, so the sixteen columns of the
// other operand are tokens: one token costs what sixteen do but for x's loads.
//
// Split.  A workgroup takes R tiles of 16 rows, its waves the chunks of the tiles
// in turn, and joins their sums in a fixed order through LDS.  E8's table (148 KB
// for 65536 points) fills a CU's LDS, so those workgroups stay, one per CU, and
// take tile after tile.  x lies in operand order (1 KB a load, whole lines): in
// place its sixteen rows often start a multiple of 4 KB apart, on the same few
// cache channels, 64 clocks a load instead of 16.
//
// Measured (microseconds at 1, 16, 32, 64, 128 tokens, bfloat16): E8 4096 x
// 14336 14.3, 18.6, 26.5, 33, 59; 4096 x 4096 8.1, 9.4, 13.6, 15.8, 27; 32768 x
// 4096 30, 33, 44, 73, 138; four bits 4096 x 14336 10.6, 15.1, 22.5, 31, 54.  An
// empty call (64 columns) is 5.7 with E8's table and 3.9 without.
#include <algorithm>
#include <type_traits>
#include "qlayer.h"

namespace mpq {

namespace {

// Sixteen waves where a wave's operands fit 128 registers, else eight.
constexpr int sk_waves(int XP, int NT, int R) { return XP * NT * R == 1 ? 16 : 8; }

struct SkinnyArgs {
  QLayer L;
  const uint16_t* x; int64_t ldx, planex;   // ldx = 0: operand order
  int kblocks;          // blocks of eight columns that x holds
  int64_t t;
  bool has_offset;
  int lut_words;
  QOut O;
};

// What a wave takes at a time: four steps (half a chunk of d = 8 codes), or a
// whole chunk of two.
constexpr int unit_steps(int f) { return q_steps(f) < 4 ? q_steps(f) : 4; }

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED, bool UNI>
__global__ __launch_bounds__(64 * sk_waves(XP, NT, R)) void q_skinny_kernel(SkinnyArgs A) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int US = unit_steps(FMT), UPC = q_steps(FMT) / US;
  constexpr int SUBS = R * NT, SK_WAVES = sk_waves(XP, NT, R);
  static_assert(SUBS <= SK_WAVES, "a wave adds up one subtile");
  // one subtile's worth of sums beside the table, or all of them over it once
  // no more tile needs it (E8), or beside it (the others' tables are small)
  constexpr bool OVER = FMT == QF_E8;
  uint32_t* lut = lds;
  v4f* red = reinterpret_cast<v4f*>(lds + (UNI ? 0 : A.lut_words));
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, kb = lane >> 4;
  const int64_t tok0 = (int64_t)blockIdx.y * (16 * NT);
  const int tgs = (A.L.tiles + R - 1) / R, units = A.L.chunks * UPC;
  // tokens past the last repeat it: a token's sums are its own column's
  const uint16_t* xrow[NT];
  const int xstep = A.ldx ? 32 : 512;   // elements from step to step
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xrow[n] = A.ldx ? A.x + min(tok0 + n * 16 + r, A.t - 1) * A.ldx + kb * 8
                    : A.x + min(tok0 / 16 + n, (A.t - 1) / 16) * ((int64_t)units * US * 512) + lane * 8;

  struct Codes {
    uint4 v[R];
  };
  struct Xs {
    v4u v[US][NT][XP];
  };
  auto load_codes = [&](Codes& c, int tg, int u) {
#pragma unroll
    for (int q = 0; q < R; ++q) {   // a tile past the last repeats it; its sums are not stored
      const char* p = reinterpret_cast<const char*>(
          A.L.packed + ((size_t)min(tg * R + q, A.L.tiles - 1) * A.L.chunks + u / UPC) * 64 + lane);
      if constexpr (UPC == 1) {
        c.v[q] = *reinterpret_cast<const uint4*>(p);
      } else {
        const uint2 h = *reinterpret_cast<const uint2*>(p + (u % UPC) * 8);
        c.v[q] = make_uint4(h.x, h.y, 0, 0);
      }
    }
  };
  // (the lanes of tokens there are not load nothing and keep their zeros, or,
  // where x is not loaded ahead, what the operand order holds for them)
  bool there[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) there[n] = tok0 + n * 16 + r < A.t;
  auto load_x = [&](Xs& x, int u, auto masked) {
    const int64_t at = (int64_t)u * US * xstep;
    const bool whole = (u + 1) * (US * 4) <= A.kblocks;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (!masked.value || there[n])
#pragma unroll
        for (int s = 0; s < US; ++s)
#pragma unroll
          for (int p = 0; p < XP; ++p) {
            const v4u* src = reinterpret_cast<const v4u*>(xrow[n] + p * A.planex + at + s * xstep);
            if (whole) {
              x.v[s][n][p] = *src;
            } else {
              x.v[s][n][p] = (v4u){0u, 0u, 0u, 0u};
              if ((u * US + s) * 4 + kb < A.kblocks) x.v[s][n][p] = *src;
            }
          }
  };
  // Codes come from HBM, a microsecond away: DEPTH units ahead.  x comes from the
  // cache, one unit ahead where the registers allow it.
  constexpr bool AHEAD = NT * XP <= 2;
  constexpr int DEPTH = SK_WAVES == 16 ? 2 : 4;
  Codes next[DEPTH];
  Xs xnext;
  if (AHEAD)
#pragma unroll
    for (int s = 0; s < US; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < XP; ++p) xnext.v[s][n][p] = (v4u){0u, 0u, 0u, 0u};
  auto load_first = [&](int tg) {
#pragma unroll
    for (int h = 0; h < DEPTH; ++h)
      if (wave + h * SK_WAVES < units) load_codes(next[h], tg, wave + h * SK_WAVES);
    if (AHEAD && wave < units) load_x(xnext, wave, std::true_type{});
  };
  load_first(blockIdx.x);
  if (!UNI) {
    q_lut_fill<FMT, T>(A.L, lut, 64 * SK_WAVES);
    __syncthreads();
  }
  const float mid = q_centre(A.L), step = UNI ? A.L.levels[1] - A.L.levels[0] : 1.f;
  constexpr bool LIFTED = UNI && !T::HALF;   // decoded entries carry Q_BASE
  const float lift = LIFTED ? Q_BASE + (float)(A.L.K / 2) : 0.f;
  for (int tg = blockIdx.x; tg < tgs; tg += gridDim.x) {
    const bool more = tg + (int)gridDim.x < tgs;
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
          sa[q][v] = A.L.scale[i];   // (times step: see below)
          so[q][v] = A.has_offset && A.L.offset ? A.L.offset[i] : 0.f;
        }
    v4f acc[R][NT], xs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xs[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < R; ++q) acc[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    for (int ub = wave; ub < units; ub += DEPTH * SK_WAVES)
#pragma unroll
    for (int h = 0; h < DEPTH; ++h) {
      const int u = ub + h * SK_WAVES;
      if (u >= units) break;
      const Codes code = next[h];
      if (u + DEPTH * SK_WAVES < units) load_codes(next[h], tg, u + DEPTH * SK_WAVES);
      Xs x;
      if (AHEAD) {
        x = xnext;
        if (u + SK_WAVES < units) load_x(xnext, u + SK_WAVES, std::true_type{});
      } else {
        load_x(x, u, std::false_type{});
      }
      constexpr bool FRESH = GROUPED || LIFTED;   // this unit's sums apart
      v4f z[R][NT], zx[NT];
      if (FRESH) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          zx[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < R; ++q) z[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
      for (int s = 0; s < US; ++s) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          v4u w;
          if constexpr (UNI) w = q_decode_uniform<FMT, T>(A.L, code.v[q], s);
          else w = q_decode<FMT, T>(A.L, lut, code.v[q], s);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              if (FRESH) z[q][n] = T::mfma(w, x.v[s][n][p], z[q][n]);
              else acc[q][n] = T::mfma(w, x.v[s][n][p], acc[q][n]);
            }
        }
        if (A.has_offset) {
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
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v) z[q][n][v] = fmaf(-lift, zx[n][v], z[q][n][v]);
      if (GROUPED) {
        const int64_t g = (int64_t)u * (US * 32) / A.L.group;   // the unit (a chunk) lies in one group
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t i = min((int64_t)(tg * R + q) * 16 + 4 * kb + v, A.L.m - 1);
            const float a = A.L.scale[i * A.L.G + g];
            const float o = fmaf(a, mid, A.L.offset ? A.L.offset[i * A.L.G + g] : 0.f);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[q][n][v] = fmaf(a * step, z[q][n][v], fmaf(o, zx[n][v], acc[q][n][v]));
          }
      } else if (LIFTED) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          xs[n] += zx[n];
#pragma unroll
          for (int q = 0; q < R; ++q) acc[q][n] += z[q][n];
        }
      }
    }
    if (more) load_first(tg + gridDim.x);
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
      if (XP > 1) {
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
  }
}

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED, bool UNI>
hipError_t launch(const SkinnyArgs& A, hipStream_t st) {
  constexpr int SK_WAVES = sk_waves(XP, NT, R);
  const int tgs = (A.L.tiles + R - 1) / R;
  const int wgs = FMT == QF_E8 ? std::min(tgs, 256) : tgs;
  const size_t table = UNI ? 0 : (size_t)A.lut_words * 4, tile = 64 * sizeof(v4f);
  const size_t shared = FMT == QF_E8 ? std::max(table + (SK_WAVES - 1) * tile, R * NT * SK_WAVES * tile)
                                     : table + R * NT * SK_WAVES * tile;
  hipLaunchKernelGGL((q_skinny_kernel<FMT, T, XP, NT, R, GROUPED, UNI>),
                     dim3((unsigned)wgs, (unsigned)((A.t + 16 * NT - 1) / (16 * NT))), dim3(64 * SK_WAVES), shared, st, A);
  return hipGetLastError();
}

template <int FMT, typename T, int XP, int NT, bool GROUPED, bool UNI>
hipError_t pick_rows(const SkinnyArgs& A, hipStream_t st) {
  // two tiles per workgroup share x's loads, once that still leaves every CU one
  if constexpr (XP == 1 && NT <= 2 && (FMT == QF_E8 || FMT == QF_NIB))
    if (A.L.tiles >= 512) return launch<FMT, T, XP, NT, 2, GROUPED, UNI>(A, st);
  return launch<FMT, T, XP, NT, 1, GROUPED, UNI>(A, st);
}

template <int FMT, typename T, int XP, bool GROUPED, bool UNI>
hipError_t pick_tokens(const SkinnyArgs& A, hipStream_t st) {
  if (A.t <= 16) return pick_rows<FMT, T, XP, 1, GROUPED, UNI>(A, st);
  if constexpr (XP == 1)
    if (A.t > 32) return pick_rows<FMT, T, XP, 4, GROUPED, UNI>(A, st);
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
    case QF_E8: return pick_tokens<QF_E8, T, XP, false, false>(A, st);
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
  A.t = t;
  A.has_offset = L.has_offset();
  A.lut_words = (q_lut_words(L.fmt, L.lut_entries) + 3) / 4 * 4;
  A.O = O;
  if (bf16) return pick_format<OpBf16, 1>(A, st);
  return planes == 2 ? pick_format<OpF16, 2>(A, st) : pick_format<OpF16, 1>(A, st);
}

}  // namespace mpq
