// The tile loop of the 16-bit matrix products (qgemm.hip says how it works and what
// bounds it), for the kernels that end it in their own ways.
#pragma once
#include <type_traits>
#include "qlayer.h"

namespace mpq {

constexpr int BK = 32;
__device__ __forceinline__ int64_t up32(int64_t x) { return (x + 31) / 32 * 32; }
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

// Where A's elements lie: a row of it after another (of the output's columns), the
// depth along a row, in blocks (operand order, as g.K says) or in rows of g.lda; or, the
// transpose of that, the depth's rows after another: in blocks (g.acols columns a
// row) or in rows of g.lda.  Then g.arows says how many rows of the depth there are
// (blocks: up to the next sixteen); those past them, up to g.K, repeat the last, and
// B holds zeros there.
enum AMode : int { A_BLOCKS = 0, A_ROWS = 1, A_T_BLOCKS = 2, A_T_ROWS = 3 };
constexpr bool a_transposed(int mode) { return mode >= A_T_BLOCKS; }

// This wave's share of the next step's rows: sixteen rows of either operand per
// load.
template <int BM, int LOADS, int AMODE>
struct Cursor {
  const char* p[LOADS];
  int pair, k;
  __device__ __forceinline__ void seek(const QGemm& g, int64_t i0, int64_t j0, int wave, const uint32_t* off, int pair_,
                                       int k_) {
    pair = pair_;
    k = k_;
    if (pair >= g.npairs) return;
    const char* a = reinterpret_cast<const char*>(g.A + g.pa[pair] * g.planeA + i0 * (AMODE == A_ROWS ? g.lda : g.K)) +
                    (size_t)k * (AMODE == A_ROWS ? BK * 2 : 1024);
    const char* b = reinterpret_cast<const char*>(g.B + g.pb[pair] * g.planeB + j0 * (g.ldb ? g.ldb : g.K)) +
                    (size_t)k * (g.ldb ? BK * 2 : 1024);
#pragma unroll
    for (int l = 0; l < LOADS; ++l) p[l] = ((wave * LOADS + l) * 16 < BM ? a : b) + (size_t)off[l] * 16;
  }
  // Straight into an LDS stage.
  __device__ __forceinline__ void fetch(const QGemm& g, int wave, const uint32_t* off, uint16_t* stage) {
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
      const int r = (wave * LOADS + l) * 16;
      q_load_lds(p[l], stage + r * BK);
      p[l] += (r < BM ? AMODE == A_BLOCKS : !g.ldb) ? 1024 : BK * 2;
    }
    ++k;
  }
};

// The same where A lies transposed (B in blocks): the operands' places in scalar
// registers, the lanes' in 32 bits beside them.
//
// The loads go without the compiler's knowledge: it takes the transposing reads, which
// are builtins, for reads of what is still on its way, and would wait for every load before
// each of them (2048 tokens, 16384 rows of 4096 columns: 270 us).  They have no register to
// write, wait_stage counts them, and stages are read after it alone.
__device__ __forceinline__ uint64_t scalar(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ void load_lds_quiet(const char* base, uint32_t off, uint32_t dst) {
  // (five wait states between a vector instruction that writes a scalar register, as
  // readfirstlane does, and a load that reads it; one after m0)
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(scalar((uint64_t)base)),
               "s"(__builtin_amdgcn_readfirstlane(dst))
               : "m0");
}
template <int BM, int LOADS, int AMODE>
struct CursorT {
  const char *a, *b;   // of the plane, of the next step
  int pair, k;
  __device__ __forceinline__ void seek(const QGemm& g, int64_t i0, int64_t j0, int wave, const uint32_t* off, int pair_,
                                       int k_) {
    pair = pair_;
    k = k_;
    if (pair >= g.npairs) return;
    a = reinterpret_cast<const char*>(g.A + g.pa[pair] * g.planeA);
    b = reinterpret_cast<const char*>(g.B + g.pb[pair] * g.planeB + j0 * g.K) + (size_t)k * 1024;
  }
  __device__ __forceinline__ void fetch(const QGemm& g, int wave, const uint32_t* off, uint16_t* stage) {
    const uint32_t to = (uint32_t)(uintptr_t)(q_lds_ptr)stage;
    // the step's rows, or the last where it is past them
    const int rows = (int)g.arows, row = min(k * BK, AMODE == A_T_BLOCKS ? (rows - 1) / 16 * 16 : rows - 1);
    const char* at = a + (AMODE == A_T_BLOCKS ? (row >> 4) * ((g.acols >> 5) * 1024) : row * (g.lda * 2));
    const bool whole = (k + 1) * BK <= rows;
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
      const int r = (wave * LOADS + l) * 16, h = r / 16 / (BM / 32);   // h: which of the step's two sixteens
      uint32_t o = off[l] * 16;
      if (r < BM && !whole) {   // its rows past the last repeat it
        if (AMODE == A_T_BLOCKS) {
          if (h == 1 && row + 16 >= rows) o -= (uint32_t)((g.acols >> 5) * 1024);
        } else {
          o -= (uint32_t)max(0, row + h * 16 + (int)((threadIdx.x & 63) >> 2) - (rows - 1)) * (uint32_t)(g.lda * 2);
        }
      }
      load_lds_quiet(r < BM ? at : b, o, to + r * (BK * 2));
    }
    b += 1024;
    ++k;
  }
};

typedef short v4s4 __attribute__((ext_vector_type(4)));
typedef uint32_t v2u2 __attribute__((ext_vector_type(2)));

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
// The same with the depth's rows in A's stage: 16 by 32 blocks, [two sixteens of rows][BM /
// 32], the halves of their rows 8 to 15 exchanged (so that the eight rows of which 32 lanes
// read one half each lie on all 64 banks).  A read hands lane l of sixteen column l of
// four rows.
template <int BM, int SM, int SN>
__device__ __forceinline__ void read_step_t(const uint16_t* stage, int wm, int wn, int r, int kb, Frags<SM, SN>& f) {
  static_assert(SM % 2 == 0, "a wave's subtiles are whole blocks");
  typedef __attribute__((address_space(3))) v4s4* lds_ptr;
  const uint16_t* Bs = stage + (BM + wn * SN * 16 + r) * BK + (kb ^ ((r >> 1) & 3)) * 8;
  const int rr = r >> 2, q = r & 3, swap = (kb & 1) * 2;
  const uint16_t* As = stage + ((kb >> 1) * (BM / 32) + wm * (SM / 2)) * 512 + ((kb & 1) * 8 + rr) * 32 + (q & 1) * 4;
  const int own = ((q >> 1) ^ swap) * 8;   // the first half's piece; the second's is two on
#pragma unroll
  for (int j = 0; j < SN; ++j) f.b[j] = *reinterpret_cast<const v4u*>(Bs + j * 16 * BK);
#pragma unroll
  for (int i = 0; i < SM; ++i) {
    uint16_t* at = const_cast<uint16_t*>(As + (i >> 1) * 512 + (own ^ (i & 1) * 16));
    const v2u2 lo = __builtin_bit_cast(v2u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at));
    const v2u2 hi = __builtin_bit_cast(v2u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 4 * 32)));
    f.a[i] = (v4u){lo[0], lo[1], hi[0], hi[1]};
  }
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
// wm WN + wn.  At the end every wave is done with the stages.  AMODE: how A lies.
template <typename T, int BM, int BN, int WM, int WN, int AMODE>
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
  const int piece = (lane & 3) ^ ((lane >> 3) & 3), tpiece = (lane & 3) ^ ((lane >> 4) & 2);
  uint32_t off[LOADS];
#pragma unroll
  for (int l = 0; l < LOADS; ++l) {
    const int r = (wave * LOADS + l) * 16;
    const bool a = r < BM;
    const int64_t lim = (a ? g.M - 1 - i0 : g.N - 1 - j0), row = a ? r : r - BM;
    // rows past the end repeat the last sixteen, or the last
    if (a && a_transposed(AMODE)) {
      const int b = r / 16, h = b / (BM / 32);
      const int64_t col = min(i0 / 32 + b % (BM / 32), (AMODE == A_T_BLOCKS ? g.acols : up32(g.M)) / 32 - 1);
      off[l] = AMODE == A_T_BLOCKS ? (uint32_t)((h * (g.acols >> 5) + col) * 64 + (lane >> 2) * 4 + tpiece)
                                   : (uint32_t)((h * 16 + (lane >> 2)) * g.lda / 8 + col * 4 + tpiece);
    } else if (a ? AMODE == A_BLOCKS : !g.ldb) off[l] = (uint32_t)(min(row / 16, lim / 16) * (g.K * 2) + (lane >> 2) * (BK / 8) + piece);
    else
      off[l] = (uint32_t)(min(row + (lane >> 2), lim) * (a ? g.lda : g.ldb) / 8 + piece);
  }

#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int j = 0; j < SN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  const int r = lane & 15, kb = lane >> 4;
#define Q_READ(stage, f)                                                                                     \
  {                                                                                                          \
    if constexpr (a_transposed(AMODE)) read_step_t<BM, SM, SN>(stage, wm, wn, r, kb, f);                     \
    else read_step<BM, SM, SN>(stage, wm, wn, r, kb, f);                                                     \
  }
  Frags<SM, SN> f0, f1;
  std::conditional_t<a_transposed(AMODE), CursorT<BM, LOADS, AMODE>, Cursor<BM, LOADS, AMODE>> at;
  at.seek(g, i0, j0, wave, off, kt0 / kts, kt0 % kts);
  // Step kt's operands are in registers when its turn begins; the barrier then
  // says that stage kt + 1 is there and that every wave has read stage kt, whose
  // place takes step kt + STAGES.  A step in the run's middle has no branch
  // between its reads and its products, so that these wait for the reads of the
  // step before alone.
  for (int s = 0; s < STAGES; ++s)
    if (kt0 + s < kt1) {
      at.fetch(g, wave, off, lds[s]);
      if (at.k == kts) at.seek(g, i0, j0, wave, off, at.pair + 1, 0);
    }
  if (kt0 + STAGES <= kt1) wait_stage<(STAGES - 1) * LOADS>(); else wait_stage<0>();
  Q_READ(lds[0], f0);
  int here = 0, kt = kt0;   // kt's stage
#define Q_STEP(cur, nxt)                                                                                     \
  {                                                                                                          \
    wait_stage<(STAGES - 2) * LOADS>();                                                                      \
    at.fetch(g, wave, off, lds[here]);                                                                       \
    here = here + 1 == STAGES ? 0 : here + 1;                                                                \
    Q_READ(lds[here], nxt);                                                                                  \
    multiply<T, SM, SN>(cur, acc);                                                                           \
    interleave<SM * SN, (a_transposed(AMODE) ? 2 : 1) * SM + SN, a_transposed(AMODE) ? 0 : LOADS>();         \
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
      at.fetch(g, wave, off, lds[here]);                                                                     \
      if (at.k == kts) at.seek(g, i0, j0, wave, off, at.pair + 1, 0);                                        \
    }                                                                                                        \
    here = here + 1 == STAGES ? 0 : here + 1;                                                                \
    if ((kt) + 1 < kt1) Q_READ(lds[here], nxt);                                                              \
    multiply<T, SM, SN>(cur, acc);                                                                           \
  }
  for (; kt < kt1; kt += 2) {
    Q_STEP(kt, f0, f1);
    if (kt + 1 < kt1) Q_STEP(kt + 1, f1, f0);
  }
#undef Q_STEP
#undef Q_READ
  wait_stage<0>();   // every read of the stages is done
}

}  // namespace mpq
