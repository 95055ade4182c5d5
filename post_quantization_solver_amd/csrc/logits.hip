// Rows of logits: token log probabilities, entropy and top alternatives, and
// distillation from a teacher's top list.
//
// Mathematics.  With c = fl(log2(e) / T) and m = max_j z_j:
//   y_j = c (z_j - m),  s = sum_j 2^y_j,  w = sum_j 2^y_j y_j,
//   lse = m + log s,  H = ln 2 (log2 s - w / s),   q_j = 2^y_j / s.
// The maximum is taken off before the scaling, so that logits masked by their
// type's lowest value stay finite.  Each 2^y is one v_exp_f32 (1 ulp), eight
// are summed as a tree and the trees in float64: a KL divergence is a small
// difference of these sums.
//
// Split.  A workgroup holds one segment of a row (at most LG_NV 16-byte vectors a
// thread) in registers: the maximum and the sums come from them.  Segments of a row
// are joined by a second kernel.
//
// Top list.  Each thread's maximum is sorted within its wave; wave w's r_w-th
// largest (sum r_w >= k over the waves) bounds the k-th largest element from
// below, so the elements at or above the smallest of those bounds hold the top
// k and are few.  The vectors that hold them are read again (of 2048 x 128256
// bfloat16, top 64, 109 MB beside the logits' 525, from beyond the L2), they go to
// LDS and are ranked by counting.  Should ties or
// masked rows make them many, a bisection over the values, then over the
// indices of equal values, finds the k exactly.
#include <math.h>
#include <algorithm>
#include <type_traits>
#include "mpq_device.h"
#include "internal.h"

namespace mpq {

namespace {

constexpr int LG_THREADS = 256;
constexpr int LG_WAVES = LG_THREADS / 64;
constexpr int LG_NV = 8;        // 16-byte vectors per thread
constexpr int LG_CAP = 2048;    // candidates in LDS
constexpr double LOG2E = 1.4426950408889634074;
constexpr double LN2 = 0.69314718055994530942;

// The storage types of logits.
struct Bf16 {
  static constexpr int VEC = 8;
  static constexpr uint32_t NEG_INF = 0xff80ff80u;
  __device__ static float elem(const uint32_t* u, int e) {
    return __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
  }
  __device__ static float load(const void* p, int64_t i) {
    return bf_bits2f(static_cast<const uint16_t*>(p)[i]);
  }
  __device__ static void store(void* p, int64_t i, float x) {
    static_cast<uint16_t*>(p)[i] = (uint16_t)f2bf_bits(x);
  }
  __device__ static uint32_t pack(float x, float y) { return f2bf_pack(x, y); }
};
struct Fp16 {
  static constexpr int VEC = 8;
  static constexpr uint32_t NEG_INF = 0xfc00fc00u;
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  __device__ static float elem(const uint32_t* u, int e) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(e & 1 ? u[e >> 1] >> 16 : u[e >> 1]));
  }
  __device__ static float load(const void* p, int64_t i) { return (float)static_cast<const _Float16*>(p)[i]; }
  __device__ static void store(void* p, int64_t i, float x) { static_cast<_Float16*>(p)[i] = (_Float16)x; }
  __device__ static uint32_t pack(float x, float y) {
    h2 v = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
};
struct Fp32 {
  static constexpr int VEC = 4;
  static constexpr uint32_t NEG_INF = 0xff800000u;
  __device__ static float elem(const uint32_t* u, int e) { return __uint_as_float(u[e]); }
  __device__ static float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  __device__ static void store(void* p, int64_t i, float x) { static_cast<float*>(p)[i] = x; }
  __device__ static uint32_t pack(float x, float) { return __float_as_uint(x); }
};

constexpr int es_of(int dtype) { return dtype == DT_F32 ? 4 : 2; }

// 16 bytes from an element-aligned address.
struct __attribute__((packed, aligned(2))) Raw16 {
  uint32_t u[4];
};
template <typename T>
__device__ __forceinline__ void load_vec(const void* row, int64_t i, int64_t end, uint32_t* u) {
  constexpr int ES = 16 / T::VEC;
  const char* p = static_cast<const char*>(row) + i * ES;
  if (i + T::VEC <= end) {
    const Raw16 r = *reinterpret_cast<const Raw16*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = r.u[q];
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = T::NEG_INF;
#pragma unroll
    for (int e = 0; e < T::VEC; ++e)
      if (i + e < end) {
        if (ES == 4) {
          u[e] = *reinterpret_cast<const uint32_t*>(p + 4 * e);
        } else {
          const uint32_t h = *reinterpret_cast<const uint16_t*>(p + 2 * e);
          u[e >> 1] = e & 1 ? (u[e >> 1] & 0xffffu) | h << 16 : (u[e >> 1] & 0xffff0000u) | h;
        }
      }
  }
}

// Elements i .. of a row, as 16 bytes (or, at its end, one by one).
template <typename T>
__device__ __forceinline__ void store_vec(char* row, int64_t i, int64_t end, const float* g) {
  if (i + T::VEC <= end) {
    Raw16 r;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r.u[q] = T::VEC == 8 ? T::pack(g[(2 * q) % T::VEC], g[(2 * q + 1) % T::VEC]) : T::pack(g[q % T::VEC], 0.f);
    *reinterpret_cast<Raw16*>(row + i * (16 / T::VEC)) = r;
  } else {
#pragma unroll
    for (int e = 0; e < T::VEC; ++e)
      if (i + e < end) T::store(row, i + e, g[e]);
  }
}

__device__ __forceinline__ float wave_max(float v) {
  for (int o = 32; o; o >>= 1) v = fmaxf(v, shfl_xor_f(v, o));
  return v;
}
// 2^y in float64 to 2^-36, by 2^n and the exponential series of f ln 2, |f| <= 1/2
// (its tenth term is below 2^-36).
__device__ __forceinline__ double exp2_series(double y) {
  y = fmax(y, -1100.0);
  const double n = rint(y), x = (y - n) * LN2;
  double p = 1.0;
#pragma unroll
  for (int k = 9; k >= 1; --k) p = fma(p * x, 1.0 / k, 1.0);
  return ldexp(p, (int)n);
}

// The tail form's s: its unlisted part as it was summed, its listed part in
// float64.  A divergence near zero is a difference that errors of the listed
// elements enter in full (of a list of one at a loss of 1e-4, 2^-13 of it), while
// an error e of the unlisted sum enters as e times the difference of the
// remainders.  Sums that are not finite stay.
__device__ __forceinline__ double tail_sum(double s, double rest, double list) {
  return s > 0.0 && s < INFINITY ? rest + list : s;
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o; o >>= 1) v += shfl_d(v, (int)(threadIdx.x & 63) ^ o);
  return v;
}
__device__ __forceinline__ int wave_sum_i(int v) {
  for (int o = 32; o; o >>= 1) v += shfl_xor_i(v, o);
  return v;
}

// max(a, b, c) without the canonicalisation of fmaxf's operands (a NaN among
// them may be dropped or win: the sums are NaN either way).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
template <typename T>
__device__ __forceinline__ float vec_max(const uint32_t* u) {
  float m = max3(T::elem(u, 0), T::elem(u, 1), T::elem(u, 2));
  if constexpr (T::VEC == 4) return max3(m, T::elem(u, 3), T::elem(u, 3));
  m = max3(m, T::elem(u, 3), T::elem(u, 4));
  m = max3(m, T::elem(u, 5), T::elem(u, 6));
  return max3(m, T::elem(u, 7), T::elem(u, 7));
}

// Keeps the compiler from carrying unpacked elements from one pass over the
// registers to the next (they would take twice the registers the raw words do).
template <int NV>
__device__ __forceinline__ void forget(uint32_t (&u)[NV][4]) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(u[j][q]));
}

// Order of floats as unsigned integers; -0 equals +0 (the caller adds +0).
__device__ __forceinline__ uint32_t ord(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unord(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Larger key = larger value, then lower index.  0 is no entry.
__device__ __forceinline__ uint64_t top_key(float x, int64_t idx) {
  return (uint64_t)ord(x + 0.f) << 32 | (uint32_t)~(uint32_t)idx;
}

// Descending bitonic sort of one float per lane.
__device__ __forceinline__ float wave_sort_desc(float v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) {
      const float o = shfl_xor_f(v, j);
      const bool up = ((lane & k) != 0) != ((lane & j) != 0);   // this lane keeps the smaller
      v = up ? fminf(v, o) : fmaxf(v, o);
    }
  return v;
}

// One segment's statistics.
struct Part {
  double s, w;      // sums of 2^y and 2^y y
  double rest;      // s without the listed entries (tail form), about mr
  float m, mr;      // the maximum; m, or the unlisted elements' own (FAR_TAIL)
};

// A sum of the unlisted elements below this share of the maximum's is taken again
// about their own maximum: float32's exponentials end at 2^-126, and 2^20 of them
// that were lost there are 2^-42 of this.  (The loss and the gradient depend on the
// unlisted elements among themselves however far they lie below the listed ones.)
constexpr double FAR_TAIL = 0x1p-64;

// A thread's sums over its vectors.  SAFE = false: y = c z - M by one fma, M =
// fl(c m); the caller takes the common c m - M out again.  It needs |M| well
// below 2^23; SAFE = true takes m off first, one more instruction an element.
// (The 0 of a logit of -inf must not be multiplied by its y.)
// MODE 0: s and w; 1: s and rest (bit e of listed(j): element e of vector j is
// listed); 2: s alone.
template <typename T, int NV, bool SAFE, int MODE, typename F>
__device__ __forceinline__ void thread_sums(const uint32_t (&u)[NV][4], int nv, float c, float m, F&& listed,
                                            double& s, double& w) {
  const float M = m * c;
  s = w = 0.0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= nv) continue;   // (the same for every thread)
    float e[T::VEC], wv = 0.f;
#pragma unroll
    for (int q = 0; q < T::VEC; ++q) {
      const float x = T::elem(u[j], q);
      const float y = SAFE ? (x - m) * c : fmaf(x, c, -M);
      e[q] = __builtin_amdgcn_exp2f(y);
      if (MODE == 0) wv = fmaf(e[q], fmaxf(y, -1e30f), wv);
    }
    if (MODE == 1) {
      const uint32_t b = listed(j);
      if (b) {   // rare
        float f[T::VEC];
#pragma unroll
        for (int q = 0; q < T::VEC; ++q) f[q] = b >> q & 1u ? 0.f : e[q];
#pragma unroll
        for (int o = T::VEC / 2; o; o >>= 1)
#pragma unroll
          for (int q = 0; q < o; ++q) f[q] += f[q + o];
        wv = f[0];
      }
#pragma unroll
      for (int o = T::VEC / 2; o; o >>= 1)
#pragma unroll
        for (int q = 0; q < o; ++q) e[q] += e[q + o];
      if (!b) wv = e[0];
    } else {
#pragma unroll
      for (int o = T::VEC / 2; o; o >>= 1)
#pragma unroll
        for (int q = 0; q < o; ++q) e[q] += e[q + o];
    }
    s += (double)e[0];
    if (MODE != 2) w += (double)wv;
    __builtin_amdgcn_sched_barrier(0);   // one vector's elements unpacked at a time
  }
}
// Whether the fma form's M resolves y.
__device__ __forceinline__ bool plain_scale(float m, float c) { return fabsf(m * c) < 0x1p20f; }

// Elements base .. end of a row that `listed` (bit e of byte v: element e of vector
// v from base on) does not name: their maximum and the sum of 2^(c (z - maximum)),
// the same in every thread.  Re-reads the row: rare.  red_m, red_s: a place per wave.
template <typename T, int THREADS>
__device__ __forceinline__ void unlisted_apart(const char* z, int64_t base, int64_t end, const uint8_t* listed,
                                               float c, float* red_m, double* red_s, float& mu, double& sum) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int at = threadIdx.x; at < (int)(end - base); at += THREADS)
      if (!(listed[at / T::VEC] >> (at % T::VEC) & 1u)) f(T::load(z, base + at));
  };
  mu = -INFINITY;
  each([&](float x) { mu = fmaxf(mu, x); });
  mu = wave_max(mu);
  __syncthreads();
  if (lane == 0) red_m[wave] = mu;
  __syncthreads();
  mu = red_m[0];
  for (int w = 1; w < THREADS / 64; ++w) mu = fmaxf(mu, red_m[w]);
  sum = 0.0;
  if (mu > -INFINITY) each([&](float x) { sum += (double)__builtin_amdgcn_exp2f((x - mu) * c); });
  sum = wave_sum(sum);
  if (lane == 0) red_s[wave] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < THREADS / 64; ++w) sum += red_s[w];
}

struct Shared {
  alignas(16) uint64_t key[LG_CAP];   // LG_CAP is a multiple of 8
  double d[2][LG_WAVES];
  float f[LG_WAVES];
  int i[LG_WAVES];
  int cnt, nvec;
  uint16_t vec[LG_NV * LG_THREADS];
};

__device__ __forceinline__ int block_count(int n, Shared& sh) {
  n = wave_sum_i(n);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.i[wave_id()] = n;
  __syncthreads();
  int a = 0;
#pragma unroll
  for (int w = 0; w < LG_WAVES; ++w) a += sh.i[w];
  return a;
}

// The k largest (value, then lowest index) of this segment, ranked, into
// list[0..k); unused places hold 0.  vm, tmax: the maxima of the thread's vectors.
template <typename T>
__device__ void segment_top(const float (&vm)[LG_NV], int nv, float tmax, const char* z, int64_t base, int64_t end,
                            int k, Shared& sh, uint64_t* __restrict__ list) {
  const int t = threadIdx.x, wave = wave_id();
  const float sorted = wave_sort_desc(tmax);
  const int act = __popcll(__ballot(tmax > -INFINITY));
  if ((t & 63) == 0) sh.i[wave] = act;
  if (t == 0) sh.cnt = sh.nvec = 0;
  __syncthreads();
  int A = 0;
#pragma unroll
  for (int w = 0; w < LG_WAVES; ++w) A += sh.i[w];
  float bound = -INFINITY;
  if (A >= k) {
    const int r = (k * act + A - 1) / A;   // <= act
    const float mine = r > 0 ? __shfl(sorted, r - 1, 64) : INFINITY;
    if ((t & 63) == 0) sh.f[wave] = mine;
    __syncthreads();
    bound = sh.f[0];
#pragma unroll
    for (int w = 1; w < LG_WAVES; ++w) bound = fminf(bound, sh.f[w]);
  }
  // the few vectors that hold such an element first, then their elements, a
  // thread each (re-read: by now many have left the L2)
#pragma unroll
  for (int j = 0; j < LG_NV; ++j) {
    if (j >= nv) break;
    if (vm[j] >= bound) sh.vec[atomicAdd(&sh.nvec, 1)] = (uint16_t)(j * LG_THREADS + t);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = t; i < sh.nvec; i += LG_THREADS) {
    const int64_t at0 = base + (int64_t)sh.vec[i] * T::VEC;
    uint32_t w[4];
    load_vec<T>(z, at0, end, w);
#pragma unroll
    for (int e = 0; e < T::VEC; ++e) {
      const float x = T::elem(w, e);
      if (x >= bound && x > -INFINITY) {
        const int at = atomicAdd(&sh.cnt, 1);
        if (at < LG_CAP) sh.key[at] = top_key(x, at0 + e);
      }
    }
  }
  __syncthreads();
  int N = sh.cnt;
  if (N > LG_CAP) {
    // bisection: the largest value with at least k elements at or above it,
    // then the index below which enough of its equals lie (re-reads the
    // segment: rare, and registers for it would halve the common case)
    auto count = [&](uint32_t v, int64_t last) {
      int n = 0;
#pragma unroll 1
      for (int64_t i = base + t; i < end; i += LG_THREADS) {
        const float x = T::load(z, i);
        const uint32_t o = ord(x + 0.f);
        n += x > -INFINITY && (o > v || (o == v && i <= last)) ? 1 : 0;
      }
      return block_count(n, sh);
    };
    uint32_t lo = ord(-INFINITY), hi = ord(INFINITY);   // count(lo) >= k, as N > LG_CAP >= k
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (count(mid, INT64_MAX) >= k) lo = mid; else hi = mid;
    }
    int64_t il = base - 1, ih = end - 1;
    while (ih - il > 1) {
      const int64_t mid = il + (ih - il) / 2;
      if (count(lo, mid) >= k) ih = mid; else il = mid;
    }
    if (t == 0) sh.cnt = 0;
    __syncthreads();
#pragma unroll 1
    for (int64_t i = base + t; i < end; i += LG_THREADS) {
      const float x = T::load(z, i);
      const uint32_t o = ord(x + 0.f);
      if (x > -INFINITY && (o > lo || (o == lo && i <= ih))) {
        const int at = atomicAdd(&sh.cnt, 1);
        if (at < LG_CAP) sh.key[at] = top_key(x, i);
      }
    }
    __syncthreads();
    N = min(sh.cnt, LG_CAP);   // k, or more where the row holds +inf (its list is not reported)
  }
  // ranks by counting, eight keys to a round (zeros fill the last)
  if (t < 8 && N + t < LG_CAP) sh.key[N + t] = 0;
  __syncthreads();
  for (int i = t; i < N; i += LG_THREADS) {
    const uint64_t key = sh.key[i];
    int rank = 0;
    for (int j = 0; j < N; j += 8) {
      ulonglong2 q[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) q[h] = reinterpret_cast<const ulonglong2*>(sh.key + j)[h];
#pragma unroll
      for (int h = 0; h < 4; ++h) rank += (q[h].x > key ? 1 : 0) + (q[h].y > key ? 1 : 0);
    }
    if (rank < k) list[rank] = key;
  }
  for (int i = N + t; i < k; i += LG_THREADS) list[i] = 0;
}

// One segment of one row: statistics, and the top list (k > 0) or the sum
// without the listed entries (TAIL).
template <typename T, bool TAIL>
__global__ __launch_bounds__(LG_THREADS) void logit_part_kernel(LogitArgs A, Part* __restrict__ parts,
                                                                uint64_t* __restrict__ lists,
                                                                float* __restrict__ zl) {
  __shared__ Shared sh;
  const int t = threadIdx.x, wave = wave_id();
  const int64_t row = blockIdx.x / A.S;
  const int seg = (int)(blockIdx.x - row * A.S);
  if (A.weights && A.weights[row] == 0.f) return;
  const int64_t base = (int64_t)seg * A.L, end = min(A.V, base + A.L);
  const char* z = static_cast<const char*>(A.z) + row * A.ldz * (16 / T::VEC);
  uint32_t u[LG_NV][4];
  const int nv = (int)((end - base + LG_THREADS * T::VEC - 1) / (LG_THREADS * T::VEC));
#pragma unroll
  for (int j = 0; j < LG_NV; ++j)
    if (j < nv) load_vec<T>(z, base + (int64_t)(j * LG_THREADS + t) * T::VEC, end, u[j]);
  // distillation: the listed logits, kept for the second kernel (which may
  // write the gradient over the logits)
  for (int i = t; i < A.k; i += LG_THREADS) {
    const int64_t id = A.ids[row * A.k + i];
    if (id >= base && id < end) zl[row * A.k + i] = T::load(z, id);
  }
  uint8_t* listed = reinterpret_cast<uint8_t*>(sh.key);   // one byte per vector
  if (TAIL) {
    for (int i = t; i < LG_NV * LG_THREADS / 4; i += LG_THREADS) reinterpret_cast<uint32_t*>(listed)[i] = 0;
    __syncthreads();
    for (int i = t; i < A.k; i += LG_THREADS) {
      const int64_t id = A.ids[row * A.k + i];
      if (id >= base && id < end) {
        const int v = (int)(id - base) / T::VEC, e = (int)(id - base) % T::VEC;
        atomicOr(reinterpret_cast<uint32_t*>(listed) + (v >> 2), 1u << (8 * (v & 3) + e));
      }
    }
  }
  float vm[LG_NV], tmax = -INFINITY;
#pragma unroll
  for (int j = 0; j < LG_NV; ++j) {
    vm[j] = -INFINITY;
    if (j < nv) vm[j] = vec_max<T>(u[j]);
    tmax = max3(tmax, vm[j], vm[j]);
  }
  float m = wave_max(tmax);
  if ((t & 63) == 0) sh.f[wave] = m;
  __syncthreads();
  m = sh.f[0];
#pragma unroll
  for (int w = 1; w < LG_WAVES; ++w) m = fmaxf(m, sh.f[w]);
  if (m == -INFINITY) m = 0.f;
  constexpr int MODE = TAIL ? 1 : 0;
  auto flags = [&](int j) -> uint32_t { return listed[j * LG_THREADS + t]; };
  double s, w;
  auto block_sums = [&]() {
    s = wave_sum(s);
    w = wave_sum(w);
    __syncthreads();
    if ((t & 63) == 0) {
      sh.d[0][wave] = s;
      sh.d[1][wave] = w;
    }
    __syncthreads();
    s = w = 0.0;
    for (int i = 0; i < LG_WAVES; ++i) {
      s += sh.d[0][i];
      w += sh.d[1][i];
    }
  };
  const bool fast = plain_scale(m, A.c);
  forget(u);
  if (fast) thread_sums<T, LG_NV, false, MODE>(u, nv, A.c, m, flags, s, w);
  else thread_sums<T, LG_NV, true, MODE>(u, nv, A.c, m, flags, s, w);
  block_sums();
  float mu = m;
  double own = 0.0;
  const bool apart = TAIL && w < FAR_TAIL && s > 0.0;   // (the same in every thread; NaN is not)
  if (apart) unlisted_apart<T, LG_THREADS>(z, base, end, listed, A.c, sh.f, sh.d[0], mu, own);
  if (t == 0) {
    Part p;
    const double d = fast ? (double)(m * A.c) - (double)m * (double)A.c : 0.0, f = exp2(d);
    p.s = s * f;
    p.w = TAIL ? 0.0 : f * (w + d * s);
    p.rest = apart ? own : w * f;
    p.m = m;
    p.mr = mu;
    parts[row * A.S + seg] = p;
  }
  if (!TAIL && A.top > 0) segment_top<T>(vm, nv, tmax, z, base, end, A.top, sh, lists + (row * A.S + seg) * A.top);
}

// Joins a row's segments, a lane each: every lane returns the row's (s, w) at the
// common m and, with TAIL, rest at mr (-inf: no unlisted element has mass).
struct RowStat {
  double s, w, rest;
  float m, mr;
};
template <bool TAIL>
__device__ RowStat join_parts(const Part* __restrict__ p, int S, float c) {
  RowStat r;
  const int lane = threadIdx.x & 63;
  float m = -INFINITY;
  for (int i = lane; i < S; i += 64)
    if (!(p[i].s == 0.0)) m = fmaxf(m, p[i].m);   // NaN sums take part
  m = wave_max(m);
  r.m = m == -INFINITY ? 0.f : m;
  r.s = r.w = r.rest = 0.0;
  r.mr = -INFINITY;
  if (TAIL) {
    for (int i = lane; i < S; i += 64)
      if (!(p[i].rest == 0.0)) r.mr = fmaxf(r.mr, p[i].mr);
    r.mr = wave_max(r.mr);
  }
  for (int i = lane; i < S; i += 64) {
    const Part q = p[i];
    if (q.s == 0.0) continue;
    const double d = ((double)q.m - (double)r.m) * (double)c, f = exp2(d);
    r.s += f * q.s;
    r.w += f * (q.w + d * q.s);
    if (TAIL && !(q.rest == 0.0)) r.rest += exp2(((double)q.mr - (double)r.mr) * (double)c) * q.rest;
  }
  r.s = wave_sum(r.s);
  r.w = wave_sum(r.w);
  if (TAIL) r.rest = wave_sum(r.rest);
  return r;
}

__device__ __forceinline__ uint64_t shfl_key(uint64_t v, int src) {
  return (uint64_t)shfl_i((uint32_t)(v >> 32), src) << 32 | shfl_i((uint32_t)v, src);
}

// A descending list of up to 64 R keys, entry 64 r + lane in register r.
template <int R>
struct TopList {
  uint64_t v[R];
  __device__ void load(const uint64_t* list, int k) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = 64 * r + (int)(threadIdx.x & 63);
      v[r] = i < k ? list[i] : 0;
    }
  }
  // The largest of this list and another: entry i against entry 64 R - 1 - i
  // leaves them as a bitonic sequence, which log2(64 R) exchanges sort.
  __device__ void merge(const TopList& o) {
    const int lane = threadIdx.x & 63;
    uint64_t b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) b[r] = shfl_key(o.v[R - 1 - r], 63 - lane);
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = max(v[r], b[r]);
    if constexpr (R == 2) {
      const uint64_t hi = max(v[0], v[1]), lo = min(v[0], v[1]);
      v[0] = hi;
      v[1] = lo;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t w = shfl_key(v[r], lane ^ d);
        v[r] = lane & d ? min(v[r], w) : max(v[r], w);
      }
  }
};

// One row: its segments' statistics joined (wave 0) and their lists merged, the
// waves each a share of them, then wave 0 the waves'.
template <typename T, int R>
__global__ __launch_bounds__(LG_THREADS) void logprob_row_kernel(LogitArgs A, const Part* __restrict__ parts,
                                                                 const uint64_t* __restrict__ lists,
                                                                 const int32_t* __restrict__ tokens,
                                                                 float* __restrict__ logprob,
                                                                 float* __restrict__ entropy, float* __restrict__ lse_out,
                                                                 int32_t* __restrict__ top_ids,
                                                                 float* __restrict__ top_lp) {
  __shared__ uint64_t keys[LG_WAVES][64 * R];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = wave_id(), waves = blockDim.x / 64;
  const int k = A.top, S = A.S;
  TopList<R> top;
  if (k > 0) {
    const uint64_t* list = lists + row * S * k;
    top.load(list + (int64_t)min(wave, S - 1) * k, wave < S ? k : 0);
    for (int g = wave + waves; g < S; g += waves) {
      TopList<R> o;
      o.load(list + (int64_t)g * k, k);
      top.merge(o);
    }
    if (waves > 1) {
#pragma unroll
      for (int r = 0; r < R; ++r) keys[wave][64 * r + lane] = top.v[r];
      __syncthreads();
      if (wave == 0)
        for (int w = 1; w < min(waves, S); ++w) {
          TopList<R> o;
          o.load(keys[w], 64 * R);
          top.merge(o);
        }
    }
  }
  if (wave > 0) return;
  const RowStat r = join_parts<false>(parts + row * S, S, A.c);
  const bool bad = !(r.s < INFINITY);   // a NaN or +inf logit
  // Log probabilities are taken of the logits as scaled by c; lse alone is
  // corrected for c's rounding: d lse / d scale is the mean logit.
  const double lg = log2(r.s);
  auto lp_of = [&](float x) {
    return bad ? NAN : x == -INFINITY ? -INFINITY : (float)((((double)x - (double)r.m) * (double)A.c - lg) * LN2);
  };
  if (lane == 0) {
    if (lse_out)
      lse_out[row] = bad         ? NAN
                     : r.s > 0.0 ? (float)((double)r.m + lg * LN2 +
                                           (1.0 - (double)A.c * LN2) * (r.w / r.s / (double)A.c))
                                 : -INFINITY;
    if (entropy) entropy[row] = bad ? NAN : r.s > 0.0 ? (float)(LN2 * (lg - r.w / r.s)) : 0.f;
    if (logprob) {
      const int32_t tok = tokens[row];
      float v = 0.f;
      if (tok >= A.V)
        v = NAN;
      else if (tok >= 0)
        v = lp_of(T::load(static_cast<const char*>(A.z) + row * A.ldz * (16 / T::VEC), tok));
      logprob[row] = v;
    }
  }
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int i = 64 * q + lane;
    if (i >= k) continue;
    const uint64_t key = top.v[q];
    if (top_ids) top_ids[row * k + i] = bad || !key ? -1 : (int32_t)~(uint32_t)key;
    if (top_lp) top_lp[row * k + i] = lp_of(key ? unord((uint32_t)(key >> 32)) : -INFINITY);
  }
}

// Distillation, one segment of one row: every workgroup joins the row's
// statistics and the teacher's list itself (k <= 128 entries), segment 0 writes
// the loss, each writes its share of the gradient: q_j times one factor per
// row, then the listed entries, each by one thread, over it.
template <typename T, bool TAIL>
__global__ __launch_bounds__(LG_THREADS) void distill_grad_kernel(LogitArgs A, const Part* __restrict__ parts,
                                                                  const float* __restrict__ zl,
                                                                  const float* __restrict__ teacher, double invT,
                                                                  float* __restrict__ loss,
                                                                  void* __restrict__ grad, int64_t ldg) {
  __shared__ int32_t sid[LG_THREADS];
  __shared__ float sp[LG_THREADS];
  __shared__ double red[3][LG_WAVES];
  __shared__ float redm[LG_WAVES];
  const int t = threadIdx.x, wave = wave_id();
  const int64_t row = blockIdx.x / A.S;
  const int seg = (int)(blockIdx.x - row * A.S);
  const float wt = A.weights ? A.weights[row] : 1.f;
  const int64_t base = (int64_t)seg * A.L, end = min(A.V, base + A.L);
  const char* z = static_cast<const char*>(A.z) + row * A.ldz * (16 / T::VEC);
  char* gr = grad ? static_cast<char*>(grad) + row * ldg * (16 / T::VEC) : nullptr;
  if (wt == 0.f) {
    if (seg == 0 && t == 0) loss[row] = 0.f;
    if (!gr) return;
    const float zero[T::VEC] = {};
    for (int64_t i = base + (int64_t)t * T::VEC; i < end; i += LG_THREADS * T::VEC) store_vec<T>(gr, i, end, zero);
    return;
  }
  const RowStat r = join_parts<TAIL>(parts + row * A.S, A.S, A.c);
  // this thread's entry of the teacher's list
  int32_t id = -1;
  double lt = -INFINITY;
  float zi = 0.f;
  if (t < A.k) {
    id = A.ids[row * A.k + t];
    if (id < 0 || id >= A.V) id = -1;
    if (id >= 0) {
      lt = (double)teacher[row * A.k + t] * invT;
      zi = zl[row * A.k + t];
      if (!TAIL && lt == -INFINITY) id = -1;   // no mass: as if not listed
    }
  }
  // p: softmax over the list, or the log probabilities themselves (tail)
  double p, lp;
  if (TAIL) {
    lp = lt;
    p = exp(lt);
  } else {
    float mx = wave_max((float)lt);
    if ((t & 63) == 0) redm[wave] = mx;
    __syncthreads();
    mx = redm[0];
    for (int i = 1; i < LG_WAVES; ++i) mx = fmaxf(mx, redm[i]);
    const double e = id >= 0 ? exp(lt - (double)mx) : 0.0;
    const double es = wave_sum(e);
    if ((t & 63) == 0) red[0][wave] = es;
    __syncthreads();
    double tot = 0.0;
    for (int i = 0; i < LG_WAVES; ++i) tot += red[0][i];
    lp = lt - (double)mx - log(tot);
    p = e / tot;
    __syncthreads();
  }
  if (id < 0) p = 0.0;
  sid[t] = id;
  sp[t] = (float)p;
  __syncthreads();
  // how often the list names each token (a token named twice has the sum)
  float pown = 0.f;
  bool first = id >= 0;
  if (id >= 0)
    for (int i = 0; i < A.k; ++i)
      if (sid[i] == id) {
        pown += sp[i];
        if (i < t) first = false;
      }
  const int named = __syncthreads_count(first ? 1 : 0);
  const double y = ((double)zi - (double)r.m) * (double)A.c;
  double s = r.s, rest = 0.0;   // rest: of s, without the listed entries
  if (TAIL) {
    if (r.mr > -INFINITY) rest = r.rest * exp2(((double)r.mr - (double)r.m) * (double)A.c);
    const double ls = wave_sum(first ? exp2_series(y) : 0.0);
    if ((t & 63) == 0) red[0][wave] = ls;
    __syncthreads();
    double list = 0.0;
    for (int i = 0; i < LG_WAVES; ++i) list += red[0][i];
    s = tail_sum(r.s, rest, list);
  }
  const double term = p == 0.0 ? 0.0 : p * (lp - (y - log2(s)) * LN2);
  const double ps = wave_sum(p), ts = wave_sum(term);
  if ((t & 63) == 0) {
    red[1][wave] = ps;
    red[2][wave] = ts;
  }
  __syncthreads();
  double psum = 0.0, kl = 0.0;
  for (int i = 0; i < LG_WAVES; ++i) {
    psum += red[1][i];
    kl += red[2][i];
  }
  const double g0 = (double)wt * invT;
  double coef = 1.0;   // of an unlisted q_j
  float mg = r.m;      // what the unlisted elements' gradients are taken about,
  double fg = 0.0;     // and their factor, where it is not coef's
  bool apart = false;
  if (TAIL) {
    // below 2^-20 the remainder is the rounding of the k float32 log
    // probabilities (k 2^-24 at most 2^-17 of them, of which most is shared);
    // a list that names every token has none
    double pt = 1.0 - psum;
    if (pt < 0x1p-20 || named >= A.V) pt = 0.0;
    if (pt > 0.0) {
      apart = rest < FAR_TAIL && s > 0.0;
      if (apart) {
        // among themselves: their gradient is q_j (1 - pt / qt), where q_j is nothing beside its share of pt
        const bool any = r.mr > -INFINITY;
        kl += pt * (log(pt) - (any ? ((double)r.mr - (double)r.m) * (double)A.c + log2(r.rest) - log2(s) : -INFINITY) * LN2);
        mg = any ? r.mr : 0.f;
        fg = any ? -g0 * pt / r.rest : 0.0;
      } else {
        const double qt = rest / s;
        kl += pt * (log(pt) - log(qt));
        coef = 1.0 - pt / qt;
      }
    }
  } else {
    coef = psum > 0.0 || psum != psum ? 1.0 : 0.0;   // an empty list teaches nothing
  }
  if (seg == 0 && t == 0) loss[row] = (float)((double)wt * kl);
  if (!gr) return;
  const float m = r.m, f = (float)(apart ? fg : coef * g0 / s), inv = (float)(1.0 / s);
  float glist = 0.f;
  if (first) glist = (__builtin_amdgcn_exp2f((zi - m) * A.c) * inv - pown) * (float)g0;
  for (int64_t i = base + (int64_t)t * T::VEC; i < end; i += LG_THREADS * T::VEC) {
    uint32_t u[4];
    load_vec<T>(z, i, end, u);
    float g[T::VEC];
#pragma unroll
    for (int e = 0; e < T::VEC; ++e) g[e] = __builtin_amdgcn_exp2f((T::elem(u, e) - mg) * A.c) * f;
    store_vec<T>(gr, i, end, g);
  }
  __syncthreads();
  if (first && id >= base && id < end) T::store(gr, id, glist);
}

// Distillation, a whole row in one workgroup's registers: read once, written
// once.  The row's last V % VEC elements, which fill no vector, are a thread's
// each.  Wave 0 takes the teacher's list (two entries a lane).
template <typename T, int THREADS, int NV, bool TAIL>
__global__ __launch_bounds__(THREADS) void distill_row_kernel(LogitArgs A, const float* __restrict__ teacher,
                                                              double invT, float* __restrict__ loss,
                                                              void* __restrict__ grad, int64_t ldg) {
  constexpr int WAVES = THREADS / 64;
  __shared__ __attribute__((aligned(16))) uint8_t listed[NV * THREADS];   // bit e of byte v: element e of vector v
  __shared__ double rs[WAVES], rw[WAVES];
  __shared__ float rm[WAVES];
  __shared__ int32_t sid[LOGIT_MAX_TOP];
  __shared__ float sp[LOGIT_MAX_TOP];
  __shared__ double s_pt, s_rest;
  __shared__ int s_twice;
  const int t = threadIdx.x, lane = t & 63, wave = wave_id();
  const int64_t row = blockIdx.x;
  const float wt = A.weights ? A.weights[row] : 1.f;
  const char* z = static_cast<const char*>(A.z) + row * A.ldz * (16 / T::VEC);
  char* gr = grad ? static_cast<char*>(grad) + row * ldg * (16 / T::VEC) : nullptr;
  const int full = (int)(A.V / T::VEC), odd = (int)(A.V % T::VEC), nv = (full + THREADS - 1) / THREADS;
  if (wt == 0.f) {
    if (t == 0) loss[row] = 0.f;
    if (!gr) return;
    const float zero[T::VEC] = {};
    for (int64_t i = (int64_t)t * T::VEC; i < A.V; i += THREADS * T::VEC) store_vec<T>(gr, i, A.V, zero);
    return;
  }
  uint32_t u[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (j < nv) {
      const int v = j * THREADS + t;
      if (v < full) {
        const Raw16 w = reinterpret_cast<const Raw16*>(z)[v];
#pragma unroll
        for (int q = 0; q < 4; ++q) u[j][q] = w.u[q];
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) u[j][q] = T::NEG_INF;
      }
    }
  const float last = t < odd ? T::load(z, (int64_t)full * T::VEC + t) : -INFINITY;
  for (int i = t; i < NV * THREADS / 16; i += THREADS) reinterpret_cast<uint4*>(listed)[i] = make_uint4(0, 0, 0, 0);
  if (t == 0) s_twice = 0;
  __syncthreads();
  // wave 0: entries lane and lane + 64 of the list (id -1: none)
  int32_t id[2] = {-1, -1};
  float zi[2] = {0.f, 0.f};
  double p[2] = {0.0, 0.0}, lp[2] = {0.0, 0.0}, ps = 0.0;
  int named = 0;
  if (wave == 0) {
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 64 * q + lane;
      if (i < A.k) {
        id[q] = A.ids[row * A.k + i];
        if (id[q] < 0 || id[q] >= A.V) id[q] = -1;
        lp[q] = (double)teacher[row * A.k + i] * invT;
        if (!TAIL && lp[q] == -INFINITY) id[q] = -1;   // no mass: as if not listed
      }
      if (id[q] >= 0) {
        zi[q] = T::load(z, id[q]);
        mx = fmaxf(mx, (float)lp[q]);
        const int v = id[q] / T::VEC, e = id[q] % T::VEC;
        const uint32_t bit = 1u << (8 * (v & 3) + e);
        if (atomicOr(reinterpret_cast<uint32_t*>(listed) + (v >> 2), bit) & bit) s_twice = 1;
        else ++named;
      }
    }
    if (TAIL) {
#pragma unroll
      for (int q = 0; q < 2; ++q) p[q] = id[q] >= 0 ? exp(lp[q]) : 0.0;
      ps = wave_sum(p[0] + p[1]);
    } else {
      mx = wave_max(mx);
#pragma unroll
      for (int q = 0; q < 2; ++q) p[q] = id[q] >= 0 ? exp(lp[q] - (double)mx) : 0.0;
      ps = wave_sum(p[0] + p[1]);
      if (ps > 0.0 || ps != ps) {
        const double l = log(ps), inv = 1.0 / ps;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          p[q] *= inv;
          lp[q] -= (double)mx + l;
        }
        ps = 1.0;
      }
    }
    named = wave_sum_i(named);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (64 * q + lane < LOGIT_MAX_TOP) {
        sid[64 * q + lane] = id[q];
        sp[64 * q + lane] = (float)p[q];
      }
    if (lane == 0) {
      // tail: the remainder (below 2^-20 it is the rounding of k float32 log
      // probabilities; a list that names every token has none); else whether
      // the list teaches anything
      double pt = ps;
      if (TAIL) {
        pt = 1.0 - ps;
        if (pt < 0x1p-20 || named >= A.V) pt = 0.0;
      }
      s_pt = pt;
    }
  }
  float m = last;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (j < nv) {
      const float v = vec_max<T>(u[j]);
      m = max3(m, v, v);
      __builtin_amdgcn_sched_barrier(0);
    }
  m = wave_max(m);
  if (lane == 0) rm[wave] = m;
  __syncthreads();
  m = rm[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) m = fmaxf(m, rm[w]);
  if (m == -INFINITY) m = 0.f;
  auto flags = [&](int j) -> uint32_t { return listed[j * THREADS + t]; };
  constexpr int MODE = TAIL ? 1 : 2;
  const bool fast = plain_scale(m, A.c);
  double s, rest;
  forget(u);
  if (fast) thread_sums<T, NV, false, MODE>(u, nv, A.c, m, flags, s, rest);
  else thread_sums<T, NV, true, MODE>(u, nv, A.c, m, flags, s, rest);
  const float M = m * A.c;
  auto two_to = [&](float x) { return __builtin_amdgcn_exp2f(fast ? fmaf(x, A.c, -M) : (x - m) * A.c); };
  const float elast = two_to(last);
  s += (double)elast;
  if (TAIL && t < odd && !(listed[full] >> t & 1u)) rest += (double)elast;
  s = wave_sum(s);
  if (TAIL) rest = wave_sum(rest);
  if (lane == 0) {
    rs[wave] = s;
    rw[wave] = rest;
  }
  __syncthreads();
  s = rest = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    s += rs[w];
    rest += rw[w];
  }
  // 2^y / s is q whatever M was rounded to: the sums carry the same factor
  const double pt = s_pt, g0 = (double)wt * invT;
  const double coef = TAIL ? (pt > 0.0 ? 1.0 - pt * s / rest : 1.0) : (pt != 0.0 ? 1.0 : 0.0);
  float f = (float)(coef * g0 / s), mg = m;
  const bool apart = TAIL && pt > 0.0 && rest < FAR_TAIL && s > 0.0;   // (the same in every thread; NaN is not)
  if (apart) {   // the unlisted elements' gradients among themselves, as in distill_grad_kernel
    float mu;
    double own;
    unlisted_apart<T, THREADS>(z, 0, A.V, listed, A.c, rm, rs, mu, own);
    const bool any = mu > -INFINITY;
    if (t == 0) s_rest = own;   // (for the loss, when the row's registers are free)
    mg = any ? mu : 0.f;
    f = any ? -(float)(g0 * pt) / (float)own : 0.f;   // (1 <= own <= 2^20)
  }
  if (gr) {
    forget(u);
    auto put = [&](auto safe) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j < nv) {
          float g[T::VEC];
#pragma unroll
          for (int e = 0; e < T::VEC; ++e) {
            const float x = T::elem(u[j], e);
            g[e] = __builtin_amdgcn_exp2f(safe.value ? (x - mg) * A.c : fmaf(x, A.c, -M)) * f;
          }
          Raw16 w;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w.u[q] = T::VEC == 8 ? T::pack(g[(2 * q) % T::VEC], g[(2 * q + 1) % T::VEC]) : T::pack(g[q % T::VEC], 0.f);
          if (j * THREADS + t < full) reinterpret_cast<Raw16*>(gr)[j * THREADS + t] = w;
          __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (fast && !apart) put(std::false_type{}); else put(std::true_type{});
    if (t < odd)
      T::store(gr, (int64_t)full * T::VEC + t, (apart ? __builtin_amdgcn_exp2f((last - mg) * A.c) : elast) * f);
  }
  __syncthreads();
  if (wave != 0) return;
  // the listed entries' gradients, over what was written there; the loss
  double y[2], list = 0.0, kl = 0.0;
  bool first[2];
  float own[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    y[q] = fast ? (double)zi[q] * (double)A.c - (double)M : ((double)zi[q] - (double)m) * (double)A.c;
    first[q] = id[q] >= 0;
    own[q] = (float)p[q];
    if (s_twice && first[q]) {   // a token named twice has the sum, and one writer
      own[q] = 0.f;
      for (int i = 0; i < A.k; ++i)
        if (sid[i] == id[q]) {
          own[q] += sp[i];
          if (i < 64 * q + lane) first[q] = false;
        }
    }
    if (TAIL && first[q]) list += exp2_series(y[q]);
  }
  if (TAIL) s = tail_sum(s, rest, wave_sum(list));
  const double lg = log2(s);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (p[q] != 0.0) kl += p[q] * (lp[q] - (y[q] - lg) * LN2);
    if (gr && first[q]) T::store(gr, id[q], (two_to(zi[q]) * (float)(1.0 / s) - own[q]) * (float)g0);
  }
  kl = wave_sum(kl);
  if (TAIL && pt > 0.0) {
    if (apart) {   // (mg is the unlisted maximum; 0, with no sum, where there is none)
      const double far = fast ? (double)mg * (double)A.c - (double)M : ((double)mg - (double)m) * (double)A.c;
      kl += pt * (log(pt) - (far + log2(s_rest) - lg) * LN2);
    } else {
      kl += pt * (log(pt) - log(rest / s));
    }
  }
  if (lane == 0) loss[row] = (float)((double)wt * kl);
}

}  // namespace

// ------------------------------------------------------------------ launchers

// Segments: at most the registers of a workgroup, and shorter where there are
// few rows, so that at least 512 workgroups (two per CU) share the work, but no
// more of them than a row has 4096 elements or a part of them.
void logit_split(LogitArgs& A) {
  const int64_t vec = 16 / es_of(A.dtype);
  const int64_t most = (int64_t)LG_NV * LG_THREADS * vec;
  const int64_t need = (A.V + most - 1) / most;
  const int64_t want = std::min((A.V + 4095) / 4096, (512 + A.t - 1) / std::max<int64_t>(A.t, 1));
  int64_t S = std::max(need, want);
  A.L = ((A.V + S - 1) / S + vec - 1) / vec * vec;
  A.S = (int)((A.V + A.L - 1) / A.L);
}

size_t logit_workspace(const LogitArgs& A) {
  const size_t rows = (size_t)A.t * A.S;
  return rows * sizeof(Part) + rows * A.top * sizeof(uint64_t) + (size_t)A.t * A.k * sizeof(float);
}

#define LOGIT_TYPES(dtype, call)      \
  switch (dtype) {                    \
    case DT_BF16: { using T = Bf16; call; break; } \
    case DT_F16: { using T = Fp16; call; break; }  \
    default: { using T = Fp32; call; break; }      \
  }

// Launches for as many rows at a time as a grid takes (fewer than 2^32 threads in
// all, of up to 1024 a workgroup): launch(those rows' arguments, the first row).
constexpr int64_t LG_LAUNCH = 1 << 21;   // workgroups

template <typename F>
static hipError_t in_slices(const LogitArgs& A, F&& launch) {
  const int64_t most = std::max<int64_t>(1, LG_LAUNCH / A.S);
  for (int64_t r0 = 0; r0 < A.t; r0 += most) {
    LogitArgs B = A;
    B.t = std::min(most, A.t - r0);
    B.z = static_cast<const char*>(A.z) + r0 * A.ldz * es_of(A.dtype);
    if (A.ids) B.ids += r0 * A.k;
    if (A.weights) B.weights += r0;
    const hipError_t e = launch(B, r0);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename P>
static P* from_row(P* p, int64_t elements) { return p ? p + elements : nullptr; }

hipError_t launch_token_logprobs(const LogitArgs& all, const int32_t* tokens, float* logprob, float* entropy,
                                 float* lse, int32_t* top_ids, float* top_lp, void* ws, hipStream_t st) {
  Part* const all_parts = static_cast<Part*>(ws);
  uint64_t* const all_lists = reinterpret_cast<uint64_t*>(all_parts + all.t * all.S);
  return in_slices(all, [&](const LogitArgs& A, int64_t r0) {
    Part* parts = all_parts + r0 * A.S;
    uint64_t* lists = all_lists + r0 * A.S * A.top;
    LOGIT_TYPES(A.dtype, hipLaunchKernelGGL((logit_part_kernel<T, false>), dim3((unsigned)(A.t * A.S)),
                                            dim3(LG_THREADS), 0, st, A, parts, lists, static_cast<float*>(nullptr)));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // one wave per row where there is little to merge
    auto rows = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)A.t), dim3(A.S > 2 && A.top > 0 ? LG_THREADS : 64), 0, st, A, parts,
                         lists, from_row(tokens, r0), from_row(logprob, r0), from_row(entropy, r0), from_row(lse, r0),
                         from_row(top_ids, r0 * A.top), from_row(top_lp, r0 * A.top));
    };
    if (A.top <= 64) {
      LOGIT_TYPES(A.dtype, (rows(logprob_row_kernel<T, 1>)));
    } else {
      LOGIT_TYPES(A.dtype, (rows(logprob_row_kernel<T, 2>)));
    }
    return hipGetLastError();
  });
}

hipError_t launch_distill(const LogitArgs& all, const float* teacher, double invT, bool tail, float* loss, void* grad,
                          int64_t ldg, void* ws, hipStream_t st) {
  Part* const all_parts = static_cast<Part*>(ws);
  float* const all_zl = reinterpret_cast<float*>(all_parts + all.t * all.S);
  // rows that fit one workgroup's registers, where there are enough of them to
  // keep half the CUs at work
  const int64_t vec = 16 / es_of(all.dtype);
  const bool whole = all.t >= 128 && all.V <= 1024 * 16 * vec, narrow = all.V <= 256 * 8 * vec;
  return in_slices(all, [&](const LogitArgs& A, int64_t r0) {
    const float* list = from_row(teacher, r0 * A.k);
    float* l = loss + r0;
    void* g = from_row(static_cast<char*>(grad), r0 * ldg * es_of(A.dtype));
    if (whole) {
      auto row = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)A.t), dim3(threads), 0, st, A, list, invT, l, g, ldg);
      };
      if (narrow && tail) {
        LOGIT_TYPES(A.dtype, (row(distill_row_kernel<T, 256, 8, true>, 256)));
      } else if (narrow) {
        LOGIT_TYPES(A.dtype, (row(distill_row_kernel<T, 256, 8, false>, 256)));
      } else if (tail) {
        LOGIT_TYPES(A.dtype, (row(distill_row_kernel<T, 1024, 16, true>, 1024)));
      } else {
        LOGIT_TYPES(A.dtype, (row(distill_row_kernel<T, 1024, 16, false>, 1024)));
      }
      return hipGetLastError();
    }
    Part* parts = all_parts + r0 * A.S;
    float* zl = all_zl + r0 * A.k;
    const dim3 grid((unsigned)(A.t * A.S)), block(LG_THREADS);
    auto part = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, st, A, parts, static_cast<uint64_t*>(nullptr), zl);
    };
    auto finish = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, st, A, parts, zl, list, invT, l, g, ldg);
    };
    if (tail) {
      LOGIT_TYPES(A.dtype, (part(logit_part_kernel<T, true>)));
    } else {
      LOGIT_TYPES(A.dtype, (part(logit_part_kernel<T, false>)));
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (tail) {
      LOGIT_TYPES(A.dtype, (finish(distill_grad_kernel<T, true>)));
    } else {
      LOGIT_TYPES(A.dtype, (finish(distill_grad_kernel<T, false>)));
    }
    return hipGetLastError();
  });
}

}  // namespace mpq
