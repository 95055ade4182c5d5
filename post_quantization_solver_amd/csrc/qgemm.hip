// 16-bit matrix products with a fused epilogue, for a solved layer's product
// with many rows and for its gradients (qlayer.h, QGemm).
//
// Workgroup tile BM x BN of the output, K in steps of 32 through four to six LDS
// stages filled by direct global -> LDS loads (16 bytes a lane), so that three to
// five steps are on their way while the matrix cores work on another out of
// registers.  A step's products stand between its loads and the LDS reads of the
// next step's operands, one each, and one barrier ends it.  A row's four 16-byte
// pieces of a step are stored permuted by the row's bits 1 and 2, so that the
// sixteen rows of an operand read spread over the banks.  Operands of more than
// 16 bits enter as planes whose sum they are: the products of plane pairs add up
// in the same float32 accumulators.
//
// Bound.  The matrix cores are busy 62 % of the time in the large tiles (2048 x
// 4096 x 14336: 198 us of the 224 of a whole call in a graph, 1.2 PFLOP/s of the
// 2.07 that they reach alone; 222 under a tracer), the rest is the step's barrier;
// the small tile waits for the L2's 64 bytes a clock and CU.  Planes are in blocks
// of 16 rows by 32 columns: rows of a matrix a multiple of 4 KB apart lie on the
// same few cache channels (before the loads stood between the products, the call
// took 293 us with planes in rows and 262 in blocks).
#include <algorithm>
#include "qgemm_tile.h"

namespace mpq {

namespace {

template <typename T, int BM, int BN, int WM, int WN, int AMODE>
__global__ __launch_bounds__(64 * WM * WN, 2) void q_gemm_kernel(QGemm g, float* __restrict__ part, int splits) {
  constexpr int WAVES = WM * WN;
  constexpr int SM = BM / WM / 16, SN = BN / WN / 16;   // 16 x 16 subtiles of a wave
  constexpr int STAGES = gemm_stages(BM, BN);
  __shared__ __attribute__((aligned(1024))) uint16_t lds[STAGES][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, kb = lane >> 4;
  int split;
  int64_t i0, j0;
  v4f acc[SM][SN];
  q_gemm_tile<T, BM, BN, WM, WN, AMODE>(g, splits, lds, acc, split, i0, j0);
  // Epilogue: sixteen rows of the output at a time through this wave's part of
  // LDS, so that a row leaves as runs of SM * 16 columns.  A lane has the same
  // four columns throughout; its rows' loads go out together.
  constexpr int PITCH = SM * 16 + 4, QUADS = SM * 4, RPI = 64 / QUADS, IT = 16 / RPI;
  static_assert(WAVES * 16 * PITCH * 4 <= (int)sizeof(lds), "the epilogue's rows fit the stages");
  float* reg = reinterpret_cast<float*>(lds[0]) + wave * 16 * PITCH;
  const int qrow = lane / QUADS, qcol = lane % QUADS * 4;
  const int64_t ii = i0 + wm * SM * 16 + qcol;
  float* own = reg + qrow * PITCH + qcol;   // and every RPI rows from there
  const QCol C = q_col4(g.O, ii);
  auto slot = [&](int it) { return reinterpret_cast<v4f*>(own + it * RPI * PITCH); };
  QLevels levels = {0.f, 0.f};
  const bool nib = g.L.fmt == QF_NIB;
  if (g.cpart) levels = q_levels(g.L);
#pragma unroll 1
  for (int j = 0; j < SN; ++j) {   // (one copy of the body; the accumulators by constant index)
#pragma unroll
    for (int jc = 0; jc < SN; ++jc)
      if (jc == j) {
#pragma unroll
        for (int i = 0; i < SM; ++i) *reinterpret_cast<v4f*>(reg + r * PITCH + i * 16 + 4 * kb) = acc[i][jc];
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int64_t jj = j0 + (wn * SN + j) * 16 + qrow;   // and every RPI rows from there
    if (g.cpart) {   // (rows past the last: of its sixteen, or of the last)
      const uint16_t* codes = q_code4_at(g.L, (g.row0 + min(j0 + (wn * SN + j) * 16, (g.N - 1) & ~(int64_t)15)) >> 4,
                                         min(ii, (g.M - 1) & ~(int64_t)3));
      uint32_t code[IT];
      float f[IT];
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int64_t row = min(jj + it * RPI, g.N - 1);
        code[it] = q_code4_of(g.L, codes, qrow + it * RPI);
        f[it] = pow2(-pow2_shift(g.O.rowmax[row]));
      }
      auto contract = [&](auto entries) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          float e[4], se = 0.f, s1 = 0.f;
          entries(code[it], e);
          const v4f x = *slot(it);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float v = k < C.live ? x[k] * C.a[k] * f[it] : 0.f;
            se = fmaf(e[k], v, se);
            s1 += v;
          }
          // sixteen lanes hold one row's 64 columns
          se += dpp_f<DPP_XOR1>(se); s1 += dpp_f<DPP_XOR1>(s1);
          se += dpp_f<DPP_XOR2>(se); s1 += dpp_f<DPP_XOR2>(s1);
          se += dpp_f<DPP_HALF_MIRROR>(se); s1 += dpp_f<DPP_HALF_MIRROR>(s1);
          se += dpp_f<DPP_MIRROR>(se); s1 += dpp_f<DPP_MIRROR>(s1);
          if ((lane & 15) == 0 && jj + it * RPI < g.N && C.live > 0)
            g.cpart[((size_t)split * g.N + jj + it * RPI) * g.cblocks + ii / Q_CONTRACT] = make_float2(se, s1);
        }
      };
      if ((g.L.fmt == QF_NIB || g.L.fmt == QF_BYTE) && g.L.uniform)   // (no branch in the loop)
        contract([&](uint32_t c, float* e) {
          c >>= nib ? 8 * (qcol >> 2 & 1) : 0;
          const uint32_t q[4] = {c, c >> 16, c >> (nib ? 4 : 8), c >> (nib ? 20 : 24)};
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = fmaf((float)(q[k] & (nib ? 15u : 63u)), levels.step, levels.base);
        });
      else
        contract([&](uint32_t c, float* e) { q_entries4(g.L, levels, c, ii, e); });
    } else if (part) {
      // rows of part are padded to four columns
#pragma unroll
      for (int it = 0; it < IT; ++it)
        if (jj + it * RPI < g.N && C.live > 0)
          *reinterpret_cast<v4f*>(part + ((size_t)split * g.N + jj + it * RPI) * ((g.M + 3) / 4 * 4) + ii) = *slot(it);
    } else if (C.live > 0) {
      float res[IT][4];
#pragma unroll
      for (int it = 0; it < IT; ++it) {
#pragma unroll
        for (int k = 0; k < 4; ++k) res[it][k] = 0.f;
        if (g.O.res && jj + it * RPI < g.N)
          load4(g.O.res, (jj + it * RPI) * g.O.ldres + ii, g.O.dtype, g.O.vec, C.live, res[it]);
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        if (jj + it * RPI >= g.N) continue;
        const v4f x = *slot(it);
        float v[4] = {x[0], x[1], x[2], x[3]};
        q_affine4(g.O, C, jj + it * RPI, v);
        if (g.O.pre) store4(g.O.pre, (jj + it * RPI) * g.O.ldpre + ii, g.O.dtype, g.O.vec, C.live, v);
        *slot(it) = (v4f){v[0], v[1], v[2], v[3]};
      }
      if (g.O.act != ACT_NONE) {   // (its code stands once)
#pragma unroll 1
        for (int it = 0; it < IT; ++it) {
          v4f x = *slot(it);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = act_fwd(g.O.act, x[k]);
          *slot(it) = x;
        }
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        if (jj + it * RPI >= g.N) continue;
        const v4f x = *slot(it);
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = x[k] + res[it][k];
        store4(g.O.y, (jj + it * RPI) * g.O.ldy + ii, g.O.dtype, g.O.vec, C.live, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// Adds the splits in order and finishes.
__global__ __launch_bounds__(256) void q_split_finish_kernel(const float* __restrict__ part, int splits, int64_t N,
                                                             int64_t Mp, QOut O) {
  const int64_t quads = Mp / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= N * quads) return;
  const int64_t j = at / quads, i = (at - j * quads) * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float4 q = *reinterpret_cast<const float4*>(part + ((size_t)s * N + j) * Mp + i);
    v[0] += q.x;
    v[1] += q.y;
    v[2] += q.z;
    v[3] += q.w;
  }
  q_finish4(O, j, i, v);
}

// Tile 256 x 256 moves the fewest bytes into LDS per product, 128 x 128 twice
// as many, where the L2's 64 bytes a clock and CU are the limit: the largest
// tile that still gives three CUs in four a workgroup is taken.  (4096 x 14336,
// whole calls: 2048 tokens 128 x 128 273 us, 256 x 128 222 us, 256 x 256 in two
// splits 238 us; 4096 tokens 553, 415, 377.)
enum Tile : int { TILE_256 = 0, TILE_256_128 = 1, TILE_128 = 2 };
struct Plan {
  int tile;
  int64_t tiles;
  int splits;
};
Plan plan(int64_t M, int64_t N, int64_t K, int npairs) {
  Plan p;
  auto count = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  p.tile = count(256, 256) >= 192 ? TILE_256 : count(256, 128) >= 192 ? TILE_256_128 : TILE_128;
  p.tiles = p.tile == TILE_256 ? count(256, 256) : p.tile == TILE_256_128 ? count(256, 128) : count(128, 128);
  const int64_t kts = K / BK * npairs;
  p.splits = 1;
  // two workgroups of the small tile fit a CU; a split keeps at least 16 steps
  if (p.tile == TILE_128 && p.tiles < 256) p.splits = (int)std::max<int64_t>(1, std::min({512 / p.tiles, kts / 16, (int64_t)16}));
  return p;
}

}  // namespace

void q_pairs(QGemm& g, int PA, int PB) {
  g.npairs = 0;
  for (int s = 0; s <= 1; ++s)
    for (int p = 0; p <= s; ++p)
      if (p < PA && s - p < PB) {
        g.pa[g.npairs] = (uint8_t)p;
        g.pb[g.npairs++] = (uint8_t)(s - p);
      }
}

int q_gemm_splits(int64_t M, int64_t N, int64_t K, int npairs) {
  return M <= 0 || N <= 0 ? 1 : plan(M, N, K, npairs).splits;
}

size_t q_gemm_workspace(int64_t M, int64_t N, int64_t K, int npairs) {
  if (M <= 0 || N <= 0) return 0;
  const Plan p = plan(M, N, K, npairs);
  return p.splits > 1 ? (size_t)p.splits * N * ((M + 3) / 4 * 4) * sizeof(float) : 0;
}

template <typename T, int AMODE>
static hipError_t run(const QGemm& g, float* part, hipStream_t st) {
  const Plan p = plan(g.M, g.N, g.K, g.npairs);
  float* out = p.splits > 1 && !g.cpart ? part : nullptr;
  const dim3 grid((unsigned)(p.tiles * p.splits));
  if (p.tile == TILE_256)
    hipLaunchKernelGGL((q_gemm_kernel<T, 256, 256, 2, 4, AMODE>), grid, dim3(512), 0, st, g, out, p.splits);
  else if (p.tile == TILE_256_128)
    hipLaunchKernelGGL((q_gemm_kernel<T, 256, 128, 4, 2, AMODE>), grid, dim3(512), 0, st, g, out, p.splits);
  else
    hipLaunchKernelGGL((q_gemm_kernel<T, 128, 128, 2, 2, AMODE>), grid, dim3(256), 0, st, g, out, p.splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !out) return e;
  const int64_t Mp = (g.M + 3) / 4 * 4;
  hipLaunchKernelGGL(q_split_finish_kernel, dim3((unsigned)((g.N * (Mp / 4) + 255) / 256)), dim3(256), 0, st, part,
                     p.splits, g.N, Mp, g.O);
  return hipGetLastError();
}

hipError_t launch_q_gemm(const QGemm& g, float* part, hipStream_t st) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  if (g.K % BK != 0 || g.K <= 0) return hipErrorInvalidValue;
  if (g.acols) return run<OpF16, A_T_BLOCKS>(g, part, st);
  if (g.lda) return g.bf16 ? run<OpBf16, A_ROWS>(g, part, st) : run<OpF16, A_ROWS>(g, part, st);
  return g.bf16 ? run<OpBf16, A_BLOCKS>(g, part, st) : run<OpF16, A_BLOCKS>(g, part, st);
}

}  // namespace mpq
