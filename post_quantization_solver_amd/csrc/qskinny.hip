// The product of a solved layer with few rows, straight from its packed codes.
//
// Mathematics.  z[i] = sum_j e_ij x_j with the codebook's entries as they are
// (exact in 16 bits) and float32 sums, then u = a z + o' sum_j x_j: no weight is
// ever formed, so none is rounded.  The sum over x rides along as one more
// matrix product, with a row of ones in the layer's place.  float32 x enters as
// two float16 terms (22 bits) of x times a power of two per token.
//
// Split.  HBM traffic is the packed codes (2 bits a weight for E8); a wave's
// matrix operand is what its lanes decode, sixteen rows at a time, so the
// sixteen columns of the other operand are tokens: one token costs what
// sixteen do.  A workgroup of 16 waves takes R tiles of 16 rows, its waves the
// chunks of the tiles in turn, and joins their sums in a fixed order through
// LDS.  E8's table (148 KB for 65536 points) fills a CU's LDS, so those
// workgroups stay, one per CU, and take tile after tile.
#include <algorithm>
#include "qlayer.h"

namespace mpq {

namespace {

constexpr int SK_WAVES = 16;

struct SkinnyArgs {
  QLayer L;
  const uint16_t* x; int64_t ldx, planex;
  int kblocks;          // blocks of eight columns that x holds
  int64_t t;
  bool has_offset;
  int lut_words;
  QOut O;
};

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED>
__global__ __launch_bounds__(64 * SK_WAVES) void q_skinny_kernel(SkinnyArgs A) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  constexpr int STEPS = q_steps(FMT);
  uint32_t* lut = lds;
  v4f* red = reinterpret_cast<v4f*>(lds + A.lut_words);   // (SK_WAVES - 1) x 64
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, kb = lane >> 4;
  q_lut_fill<FMT, T>(A.L, lut, 64 * SK_WAVES);
  __syncthreads();
  const int64_t tok0 = (int64_t)blockIdx.y * (16 * NT);
  const float mid = q_centre(A.L);
  const int tgs = (A.L.tiles + R - 1) / R;
  for (int tg = blockIdx.x; tg < tgs; tg += gridDim.x) {
    v4f acc[R][NT], xs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xs[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < R; ++q) acc[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    const uint4* src[R];
#pragma unroll
    for (int q = 0; q < R; ++q)   // a tile past the last repeats it; its sums are not stored
      src[q] = A.L.packed + ((size_t)min(tg * R + q, A.L.tiles - 1) * A.L.chunks) * 64 + lane;
    uint4 next[R];
    if (wave < A.L.chunks)
#pragma unroll
      for (int q = 0; q < R; ++q) next[q] = src[q][(size_t)wave * 64];
    for (int c = wave; c < A.L.chunks; c += SK_WAVES) {
      uint4 code[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        code[q] = next[q];
        if (c + SK_WAVES < A.L.chunks) next[q] = src[q][(size_t)(c + SK_WAVES) * 64];
      }
      v4f z[R][NT], zx[NT];
      if (GROUPED) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          zx[n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < R; ++q) z[q][n] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
      }
      const int blk0 = c * STEPS * 4 + kb;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        v4u xf[NT][XP];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int64_t tok = tok0 + n * 16 + r;
          const bool ok = tok < A.t && blk0 + s * 4 < A.kblocks;
#pragma unroll
          for (int p = 0; p < XP; ++p) {
            xf[n][p] = (v4u){0u, 0u, 0u, 0u};
            if (ok)
              xf[n][p] = *reinterpret_cast<const v4u*>(A.x + p * A.planex + tok * A.ldx + (int64_t)(blk0 + s * 4) * 8);
          }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const v4u w = q_decode<FMT, T>(A.L, lut, code[q], s);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              if (GROUPED) z[q][n] = T::mfma(w, xf[n][p], z[q][n]);
              else acc[q][n] = T::mfma(w, xf[n][p], acc[q][n]);
            }
        }
        if (A.has_offset) {
          const v4u one = {T::ONES, T::ONES, T::ONES, T::ONES};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              if (GROUPED) zx[n] = T::mfma(one, xf[n][p], zx[n]);
              else xs[n] = T::mfma(one, xf[n][p], xs[n]);
            }
        }
      }
      if (GROUPED) {
        const int64_t g = (int64_t)c * q_chunk(FMT) / A.L.group;   // the chunk lies in one group
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t i = min((int64_t)(tg * R + q) * 16 + 4 * kb + v, A.L.m - 1);
            const float a = A.L.scale[i * A.L.G + g];
            const float o = fmaf(a, mid, A.L.offset ? A.L.offset[i * A.L.G + g] : 0.f);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[q][n][v] = fmaf(a, z[q][n][v], fmaf(o, zx[n][v], acc[q][n][v]));
          }
      }
    }
    if (!GROUPED) {
#pragma unroll
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t i = min((int64_t)(tg * R + q) * 16 + 4 * kb + v, A.L.m - 1);
          const float a = A.L.scale[i];
          const float o = A.has_offset ? fmaf(a, mid, A.L.offset ? A.L.offset[i] : 0.f) : 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[q][n][v] = fmaf(a, acc[q][n][v], A.has_offset ? o * xs[n][v] : 0.f);
        }
    }
    // Subtile (q, n) is added up, in the order of the waves, by wave (q NT + n).
    float mine[4] = {0.f, 0.f, 0.f, 0.f};
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
    if (wave < R * NT) {
      const int64_t tok = tok0 + wave % NT * 16 + r;
      if (XP > 1 && tok < A.t) {
        const float f = pow2(-pow2_shift(A.O.rowmax[tok]));
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[k] *= f;
      }
      q_finish4(A.O, tok, (int64_t)(tg * R + wave / NT) * 16 + 4 * kb, mine, false);
    }
  }
}

template <int FMT, typename T, int XP, int NT, int R, bool GROUPED>
hipError_t launch(const SkinnyArgs& A, hipStream_t st) {
  const int tgs = (A.L.tiles + R - 1) / R;
  const int wgs = FMT == QF_E8 ? std::min(tgs, 256) : tgs;
  const size_t shared = (size_t)A.lut_words * 4 + (SK_WAVES - 1) * 64 * sizeof(v4f);
  hipLaunchKernelGGL((q_skinny_kernel<FMT, T, XP, NT, R, GROUPED>),
                     dim3((unsigned)wgs, (unsigned)((A.t + 16 * NT - 1) / (16 * NT))), dim3(64 * SK_WAVES), shared, st, A);
  return hipGetLastError();
}

template <int FMT, typename T, int XP, int NT, bool GROUPED>
hipError_t pick_rows(const SkinnyArgs& A, hipStream_t st) {
  // two tiles per workgroup share x's loads, once that still leaves every CU one
  if constexpr (XP == 1 && NT <= 2 && (FMT == QF_E8 || FMT == QF_NIB))
    if (A.L.tiles >= 512) return launch<FMT, T, XP, NT, 2, GROUPED>(A, st);
  return launch<FMT, T, XP, NT, 1, GROUPED>(A, st);
}

template <int FMT, typename T, int XP, bool GROUPED>
hipError_t pick_tokens(const SkinnyArgs& A, hipStream_t st) {
  if (A.t <= 16) return pick_rows<FMT, T, XP, 1, GROUPED>(A, st);
  if constexpr (XP == 1 && !GROUPED)   // (the others' sums of 64 tokens do not fit 128 registers)
    if (A.t > 32) return pick_rows<FMT, T, XP, 4, GROUPED>(A, st);
  return pick_rows<FMT, T, XP, 2, GROUPED>(A, st);
}

template <typename T, int XP>
hipError_t pick_format(const SkinnyArgs& A, hipStream_t st) {
  const bool grouped = A.L.G > 1;
  switch (A.L.fmt) {
    case QF_NIB: return grouped ? pick_tokens<QF_NIB, T, XP, true>(A, st) : pick_tokens<QF_NIB, T, XP, false>(A, st);
    case QF_BYTE: return grouped ? pick_tokens<QF_BYTE, T, XP, true>(A, st) : pick_tokens<QF_BYTE, T, XP, false>(A, st);
    case QF_E8: return pick_tokens<QF_E8, T, XP, false>(A, st);
    default: return pick_tokens<QF_VEC, T, XP, false>(A, st);
  }
}

}  // namespace

bool q_skinny_ok(const QLayer& L) { return L.G == 1 || L.group % q_chunk(L.fmt) == 0; }

hipError_t launch_q_skinny(const QLayer& L, const uint16_t* x, int64_t ldx, int64_t planex, int kblocks, int64_t t,
                           int planes, bool bf16, const QOut& O, hipStream_t st) {
  SkinnyArgs A;
  A.L = L;
  A.x = x;
  A.ldx = ldx;
  A.planex = planex;
  A.kblocks = kblocks;
  A.t = t;
  A.has_offset = L.has_offset();
  A.lut_words = (q_lut_words(L.fmt, L.lut_entries) + 3) / 4 * 4;
  A.O = O;
  if (bf16) return pick_format<OpBf16, 1>(A, st);
  return planes == 2 ? pick_format<OpF16, 2>(A, st) : pick_format<OpF16, 1>(A, st);
}

}  // namespace mpq
