// The tile loop of the 16-bit matrix products (qgemm.hip says how it works and what
// bounds it), for the kernels that end it in their own ways.
#pragma once
#include "qlayer.h"

namespace mpq {

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
template <int BM, int LOADS, bool AROWS>
struct Cursor {
  const char* p[LOADS];
  int pair, k;
  __device__ __forceinline__ void seek(const QGemm& g, int64_t i0, int64_t j0, int wave, const uint32_t* off, int pair_,
                                       int k_) {
    pair = pair_;
    k = k_;
    if (pair >= g.npairs) return;
    const char* a = reinterpret_cast<const char*>(g.A + g.pa[pair] * g.planeA + i0 * (AROWS ? g.lda : g.K)) +
                    (size_t)k * (AROWS ? BK * 2 : 1024);
    const char* b = reinterpret_cast<const char*>(g.B + g.pb[pair] * g.planeB + j0 * (g.ldb ? g.ldb : g.K)) +
                    (size_t)k * (g.ldb ? BK * 2 : 1024);
#pragma unroll
    for (int l = 0; l < LOADS; ++l) p[l] = ((wave * LOADS + l) * 16 < BM ? a : b) + (size_t)off[l] * 16;
  }
};

// Straight into an LDS stage.
template <int BM, int LOADS, bool AROWS>
__device__ __forceinline__ void fetch_step(Cursor<BM, LOADS, AROWS>& c, const QGemm& g, int64_t i0, int64_t j0, int wave,
                                           const uint32_t* off, uint16_t* stage) {
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int r = (wave * LOADS + l) * 16;
    q_load_lds(c.p[l], stage + r * BK);
    c.p[l] += (r < BM ? !AROWS : !g.ldb) ? 1024 : BK * 2;
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

// Which tile this workgroup has, and its products summed up: D[j0 + (wn SN + b) 16 +
// lane % 16][i0 + (wm SM + a) 16 + 4 (lane / 16) + k] = acc[a][b][k], with wave
// wm WN + wn.  At the end every wave is done with the stages.  AROWS: A stays in rows of
// g.lda elements (as B in rows of g.ldb).
template <typename T, int BM, int BN, int WM, int WN, bool AROWS = false>
__device__ __forceinline__ void q_gemm_tile(const QGemm& g, int splits, uint16_t (&lds)[gemm_stages(BM, BN)][(BM + BN) * BK],
                                            v4f (&acc)[BM / WM / 16][BN / WN / 16], int& split, int64_t& i0, int64_t& j0) {
  constexpr int WAVES = WM * WN;
  constexpr int SM = BM / WM / 16, SN = BN / WN / 16;   // 16 x 16 subtiles of a wave
  constexpr int LOADS = (BM + BN) / 16 / WAVES;         // 1 KB loads per wave and step
  constexpr int STAGES = gemm_stages(BM, BN);
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / WN, wn = wave % WN;
  // tiles: contiguous runs per XCD (workgroups go to the 8 XCDs in turn), and
  // within a run groups of 8 tile rows column by column
  const int tm = (int)((g.M + BM - 1) / BM), tn = (int)((g.N + BN - 1) / BN);
  const int T_ = tm * tn;
  split = (int)(blockIdx.x / T_);
  int tile = (int)(blockIdx.x % T_);
  {
    const int per = T_ / 8, rem = T_ % 8, x = tile % 8, q = tile / 8;
    tile = x * per + min(x, rem) + q;
  }
  const int grp = tile / (8 * tn), first = grp * 8, gm = min(tm - first, 8);
  const int in = tile - grp * 8 * tn;
  i0 = (int64_t)(first + in % gm) * BM;
  j0 = (int64_t)(in / gm) * BN;

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
    if (a ? !AROWS : !g.ldb) off[l] = (uint32_t)(min(row / 16, lim / 16) * (g.K * 2) + (lane >> 2) * (BK / 8) + piece);
    else off[l] = (uint32_t)(min(row + (lane >> 2), lim) * (a ? g.lda : g.ldb) / 8 + piece);
  }

#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int j = 0; j < SN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  const int r = lane & 15, kb = lane >> 4;
  Frags<SM, SN> f0, f1;
  Cursor<BM, LOADS, AROWS> at;
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
}

}  // namespace mpq
