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
#include "qlayer.h"

namespace mpq {

namespace {

constexpr int BK = 32;
constexpr int gemm_stages(int BM, int BN) { return BM + BN <= 256 ? 4 : BM + BN <= 384 ? 6 : 5; }

// Waits until at most N of this wave's global -> LDS loads are on their way,
// and for its LDS reads; then for the workgroup.  (The builtin, so that the
// compiler knows that the reads are there and puts no wait of its own before the
// products.)
template <int N>
__device__ __forceinline__ void wait_stage() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);   // the products before stay before
  __builtin_amdgcn_s_waitcnt(q_waitcnt(N));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// This wave's share of the next step's rows: sixteen rows of either operand per
// load.
template <int BM, int LOADS>
struct Cursor {
  const char* p[LOADS];
  int pair, k;
  __device__ __forceinline__ void seek(const QGemm& g, int64_t i0, int64_t j0, int wave, const uint32_t* off, int pair_,
                                       int k_) {
    pair = pair_;
    k = k_;
    if (pair >= g.npairs) return;
    const char* a = reinterpret_cast<const char*>(g.A + g.pa[pair] * g.planeA + i0 * g.K) + (size_t)k * 1024;
    const char* b = reinterpret_cast<const char*>(g.B + g.pb[pair] * g.planeB + j0 * (g.ldb ? g.ldb : g.K)) +
                    (size_t)k * (g.ldb ? BK * 2 : 1024);
#pragma unroll
    for (int l = 0; l < LOADS; ++l) p[l] = ((wave * LOADS + l) * 16 < BM ? a : b) + (size_t)off[l] * 16;
  }
};

// Straight into an LDS stage.
template <int BM, int LOADS>
__device__ __forceinline__ void fetch_step(Cursor<BM, LOADS>& c, const QGemm& g, int64_t i0, int64_t j0, int wave,
                                           const uint32_t* off, uint16_t* stage) {
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int r = (wave * LOADS + l) * 16;
    q_load_lds(c.p[l], stage + r * BK);
    c.p[l] += r < BM || !g.ldb ? 1024 : BK * 2;
  }
  ++c.k;
}

// One wave's operands of a step.
template <int SM, int SN>
struct Frags {
  v4u a[SM], b[SN];
};
template <int BM, int SM, int SN>
__device__ __forceinline__ void read_step(const uint16_t* stage, int wm, int wn, int r, int kb, Frags<SM, SN>& f) {
  const int pc = (kb ^ ((r >> 1) & 3)) * 8;
  const uint16_t* As = stage + (wm * SM * 16 + r) * BK + pc;
  const uint16_t* Bs = stage + (BM + wn * SN * 16 + r) * BK + pc;
#pragma unroll
  for (int j = 0; j < SN; ++j) f.b[j] = *reinterpret_cast<const v4u*>(Bs + j * 16 * BK);
#pragma unroll
  for (int i = 0; i < SM; ++i) f.a[i] = *reinterpret_cast<const v4u*>(As + i * 16 * BK);
}
template <typename T, int SM, int SN>
__device__ __forceinline__ void multiply(const Frags<SM, SN>& f, v4f (&acc)[SM][SN]) {
#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int j = 0; j < SN; ++j) acc[i][j] = T::mfma(f.a[i], f.b[j], acc[i][j]);
}

// A step's instructions in turn: loads and reads go out between the products.
template <int MFMAS, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
  constexpr int MFMA = 0x8, VMEM = 0x10, DS_READ = 0x100;
  static_assert(READS + LOADS <= MFMAS, "a product before each");
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {
    __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
    __builtin_amdgcn_sched_group_barrier(VMEM, 1, 0);
  }
#pragma unroll
  for (int k = 0; k < READS; ++k) {
    __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
    __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(MFMA, MFMAS - READS - LOADS, 0);
}

template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void q_gemm_kernel(QGemm g, float* __restrict__ part, int splits) {
  constexpr int WAVES = WM * WN;
  constexpr int SM = BM / WM / 16, SN = BN / WN / 16;   // 16 x 16 subtiles of a wave
  constexpr int LOADS = (BM + BN) / 16 / WAVES;         // 1 KB loads per wave and step
  constexpr int STAGES = gemm_stages(BM, BN);
  __shared__ __attribute__((aligned(1024))) uint16_t lds[STAGES][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / WN, wn = wave % WN;
  // tiles: contiguous runs per XCD (workgroups go to the 8 XCDs in turn), and
  // within a run groups of 8 tile rows column by column
  const int tm = (int)((g.M + BM - 1) / BM), tn = (int)((g.N + BN - 1) / BN);
  const int T_ = tm * tn;
  const int split = (int)(blockIdx.x / T_);
  int tile = (int)(blockIdx.x % T_);
  {
    const int per = T_ / 8, rem = T_ % 8, x = tile % 8, q = tile / 8;
    tile = x * per + min(x, rem) + q;
  }
  const int grp = tile / (8 * tn), first = grp * 8, gm = min(tm - first, 8);
  const int in = tile - grp * 8 * tn;
  const int64_t i0 = (int64_t)(first + in % gm) * BM, j0 = (int64_t)(in / gm) * BN;

  const int kts = (int)(g.K / BK), all = kts * g.npairs;
  const int kt0 = (int)((int64_t)all * split / splits), kt1 = (int)((int64_t)all * (split + 1) / splits);

  // this lane's offsets within the tile's rows, in 16 bytes (a tile's 256 rows of
  // 2^24 columns are 8 GB)
  const int piece = (lane & 3) ^ ((lane >> 3) & 3);
  uint32_t off[LOADS];
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int r = (wave * LOADS + l) * 16;
    const bool a = r < BM;
    const int64_t lim = (a ? g.M - 1 - i0 : g.N - 1 - j0), row = a ? r : r - BM;
    // rows past the end repeat the last sixteen, or the last
    if (a || !g.ldb) off[l] = (uint32_t)(min(row / 16, lim / 16) * (g.K * 2) + (lane >> 2) * (BK / 8) + piece);
    else off[l] = (uint32_t)(min(row + (lane >> 2), lim) * g.ldb / 8 + piece);
  }

  v4f acc[SM][SN];
#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int j = 0; j < SN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  const int r = lane & 15, kb = lane >> 4;
  Frags<SM, SN> f0, f1;
  Cursor<BM, LOADS> at;
  at.seek(g, i0, j0, wave, off, kt0 / kts, kt0 % kts);
  // Step kt's operands are in registers when its turn begins; the barrier then
  // says that stage kt + 1 is there and that every wave has read stage kt, whose
  // place takes step kt + STAGES.  A step in the run's middle has no branch
  // between its reads and its products, so that these wait for the reads of the
  // step before alone.
  for (int s = 0; s < STAGES; ++s)
    if (kt0 + s < kt1) {
      fetch_step(at, g, i0, j0, wave, off, lds[s]);
      if (at.k == kts) at.seek(g, i0, j0, wave, off, at.pair + 1, 0);
    }
  if (kt0 + STAGES <= kt1) wait_stage<(STAGES - 1) * LOADS>(); else wait_stage<0>();
  read_step<BM, SM, SN>(lds[0], wm, wn, r, kb, f0);
  int here = 0, kt = kt0;   // kt's stage
#define Q_STEP(cur, nxt)                                                                                     \
  {                                                                                                          \
    wait_stage<(STAGES - 2) * LOADS>();                                                                      \
    fetch_step(at, g, i0, j0, wave, off, lds[here]);                                                         \
    here = here + 1 == STAGES ? 0 : here + 1;                                                                \
    read_step<BM, SM, SN>(lds[here], wm, wn, r, kb, nxt);                                                    \
    multiply<T, SM, SN>(cur, acc);                                                                           \
    interleave<SM * SN, SM + SN, LOADS>();                                                                   \
    if (at.k == kts) at.seek(g, i0, j0, wave, off, at.pair + 1, 0);                                          \
  }
  for (; kt + STAGES + 1 < kt1; kt += 2) {
    Q_STEP(f0, f1);
    Q_STEP(f1, f0);
  }
#undef Q_STEP
#define Q_STEP(kt, cur, nxt)                                                                                 \
  {                                                                                                          \
    if ((kt) + STAGES <= kt1) wait_stage<(STAGES - 2) * LOADS>(); else wait_stage<0>();                      \
    if ((kt) + STAGES < kt1) {                                                                               \
      fetch_step(at, g, i0, j0, wave, off, lds[here]);                                                       \
      if (at.k == kts) at.seek(g, i0, j0, wave, off, at.pair + 1, 0);                                        \
    }                                                                                                        \
    here = here + 1 == STAGES ? 0 : here + 1;                                                                \
    if ((kt) + 1 < kt1) read_step<BM, SM, SN>(lds[here], wm, wn, r, kb, nxt);                                \
    multiply<T, SM, SN>(cur, acc);                                                                           \
  }
  for (; kt < kt1; kt += 2) {
    Q_STEP(kt, f0, f1);
    if (kt + 1 < kt1) Q_STEP(kt + 1, f1, f0);
  }
#undef Q_STEP
  wait_stage<0>();   // every read of the stages is done
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
    if (g.cpart) {
      uint32_t code[IT];
      float f[IT];
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int64_t row = min(jj + it * RPI, g.N - 1);
        code[it] = q_code4(g.L, g.row0 + row, min(ii, (g.M - 1) & ~(int64_t)3));
        f[it] = pow2(-pow2_shift(g.O.rowmax[row]));
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        float e[4], se = 0.f, s1 = 0.f;
        q_entries4(g.L, code[it], ii, e);
        const v4f x = *slot(it);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < C.live) {
            const float v = x[k] * C.a[k] * f[it];
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

template <typename T>
static hipError_t run(const QGemm& g, float* part, hipStream_t st) {
  const Plan p = plan(g.M, g.N, g.K, g.npairs);
  float* out = p.splits > 1 && !g.cpart ? part : nullptr;
  const dim3 grid((unsigned)(p.tiles * p.splits));
  if (p.tile == TILE_256)
    hipLaunchKernelGGL((q_gemm_kernel<T, 256, 256, 2, 4>), grid, dim3(512), 0, st, g, out, p.splits);
  else if (p.tile == TILE_256_128)
    hipLaunchKernelGGL((q_gemm_kernel<T, 256, 128, 4, 2>), grid, dim3(512), 0, st, g, out, p.splits);
  else
    hipLaunchKernelGGL((q_gemm_kernel<T, 128, 128, 2, 2>), grid, dim3(256), 0, st, g, out, p.splits);
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
  return g.bf16 ? run<OpBf16>(g, part, st) : run<OpF16>(g, part, st);
}

}  // namespace mpq
