// One AdamW step over many tensors at once, moments in 32 or in 8 bits.
//
// Mathematics.  With g' = factor g, factor the loss scale's inverse times the
// clipping of the gradients' common norm, and t the step's number from 1 on:
//   m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
//   p' = p - lr wd p - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps).
// 8 bits: 256 elements share a float32 scale each for m and for r = sqrt(v).  A
// code is a small floating-point number of 4 exponent and 3 (m, beside its sign)
// or 4 (r) fraction bits, in units of the scale: 0 .. 2^F - 1 as they are, then
// (2^F + f) 2^(E - 1); the block's largest has the largest code.  An element is
// rounded up with the probability of where it (of a root, its square: v is what is
// kept on average) lies between two codes: to the nearest, no increment below
// half a code's step (1 - b2 of v is a thousandth, a step some tenth) would ever be
// kept.  A root that is not zero is never
// rounded to zero, which would leave its m over eps.  16-bit parameters are
// rounded the same way, for the same reason.  The random bits are a hash of
// (seed, t, the element's place in the moments).
//
// Roundings.  8-bit moments are computed in float64 up to their codes, each product
// and sum rounded as the formulas stand (an element next to a border, and a scale
// half way between two floats, which decimal betas often make, fall to the side that
// the formula says); what the parameter takes of them, and 32-bit moments, in float32.
//
// Split.  A unit is 2048 elements of one tensor, a workgroup's turn; a table
// says which tensor a unit is of.  The gradients' addresses, which change with
// every step, come as kernel arguments: as many as 440 tensors a launch.  The
// last workgroup to end counts the step, and in the norm's kernel adds up the
// others' sums, in a fixed order: no further launch.
//
// Bound.  32 bits: memory (15 million float16 parameters, 22 bytes an element, read and written: 54 us,
// 6 TB/s, some of it from the last-level cache).  8 bits: vector instructions (43.8 million bfloat16
// parameters, 10 bytes an element: 170 us, 110 instructions an element, busy 79 % of the clocks;
// 77 us at a copy's rate).  The norm reads at 3 TB/s (its waves wait for memory 91 % of the time), the moments' decoder reads and writes at
// 5.4.  A few small tensors: one launch, 4 us.
#include <math.h>
#include <type_traits>
#include "internal.h"
#include "adamw.h"
#include "qlayer.h"

namespace mpq {

namespace {

constexpr int UNIT = 2048, THREADS = 256, PER = UNIT / THREADS;

struct GradList {
  const void* p[ADAMW_LAUNCH];
};

__host__ __device__ constexpr uint32_t mix(uint32_t x) {
  // (shifts, and products with the fractions of the roots of 2 and 3)
  x ^= x >> 16;
  x *= 0x6a09e667u;
  x ^= x >> 15;
  x *= 0xbb67ae85u;
  return x ^ x >> 16;
}

// ------------------------------------------------------------------ 8-bit codes

// Units of the scale that the largest code stands for.
template <int F>
constexpr double top_value() { return (double)((2 << F) - 1) * 16384.0; }

// What a code stands for, in units of its scale.  A code's bits are a float's
// exponent and leading fraction bits; the codes below 2^F, evenly spaced like the
// 2^F after them, come as those less 2^F.
template <int F>
__device__ __forceinline__ double code_value(uint32_t c) {
  const bool low = c < 1u << F;
  const float x = __uint_as_float(((low ? c + (1u << F) : c) + ((126u + F) << F)) << (23 - F));
  return (double)(low ? x - (float)(1 << F) : x);
}
// |m| in units of the scale as a code: up where its rest and u = (h + 1/2) / 2^16 are 1
// and more together (a code is the double's leading bits; u is added below them).
__device__ __forceinline__ uint32_t code_of_mean(double x, uint32_t h) {
  const bool low = x < 8.0;
  const uint32_t hi = (uint32_t)__double2hiint(low ? x + 8.0 : x) + 2 * h + 1;
  return min((hi >> 17) - (1025u << 3) - (low ? 8u : 0u), 127u);
}
// A root's code, by where its square y (in units of the scale's) lies between the codes'
// squares: those are what has to be kept on average (by the roots, each rounding would add
// its variance to v).  The code 16 e + M stands for M 2^e (M from 16 on where e > 0), and in
// units of 2^(2 e - 17) its square, and the square where rounding up begins, are whole
// numbers.  M and e come from float32's root: next to a code that may be one off, and the
// comparison then goes the same way (u is no nearer to 0 or 1 than 2^-17).
__device__ __forceinline__ uint32_t code_of_root(double y, uint32_t h) {
  const float x = __builtin_amdgcn_sqrtf((float)y);
  const int e = max(__builtin_amdgcn_frexp_expf(x) - 5, 0);
  const uint32_t M = (uint32_t)ldexpf(x, -e);
  const uint32_t up = (M * M << 17) + __umul24(131071u - 2u * h, 2u * M + 1u);
  const uint32_t c = (uint32_t)(e << 4) + M;
  return min(__builtin_amdgcn_ldexp(y, 17 - 2 * e) >= (double)up ? c + 1 : c, 255u);
}

// What the codes of m (with their sign) and of the root stand for, for decoding: in LDS.
struct CodeTables {
  double m[256], r[256];
};
__device__ __forceinline__ void fill_tables(CodeTables& T) {
  static_assert(THREADS == 256, "a code a thread");
  const uint32_t c = threadIdx.x;
  const double v = code_value<3>(c & 127u);
  T.m[c] = c & 128u ? -v : v;
  T.r[c] = code_value<4>(c);
}

// ------------------------------------------------------------------ memory

// Eight consecutive elements from p[i] on, as many as live (FULL: all, from aligned
// addresses: no load under a branch, so that they are on their way together).
template <bool FULL>
__device__ __forceinline__ void load8(const void* p, int64_t i, int dtype, int live, float* v) {
  if constexpr (FULL) {
    if (dtype == DT_F32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = q[0], b = q[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu;
        v[k] = dtype == DT_BF16 ? OpBf16::val(b) : OpF16::val(b);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < live ? load_as_f32(p, i + k, dtype) : 0.f;
  }
}

// A parameter's 16 bits, rounded by 16 random ones; what is not finite as it is,
// float16 below its normal range to the nearest.
__device__ __forceinline__ uint32_t round16(float x, int dtype, uint32_t h) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7f800000u) == 0x7f800000u) return dtype == DT_BF16 ? OpBf16::bits(x) : OpF16::bits(x);
  if (dtype == DT_BF16) return (b + (h & 0xffffu)) >> 16;
  return OpF16::bits(__uint_as_float((b + (h & 0x1fffu)) & ~0x1fffu));
}
template <bool FULL>
__device__ __forceinline__ void store8(void* p, int64_t i, int dtype, int live, const float* v, const uint32_t* h) {
  if (dtype == DT_F32) {
    float* q = static_cast<float*>(p) + i;
    if constexpr (FULL) {
      reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < live) q[k] = v[k];
    }
    return;
  }
  uint16_t* q = static_cast<uint16_t*>(p) + i;
  uint32_t b[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) b[k] = round16(v[k], dtype, h[k]);
  if constexpr (FULL) {
    *reinterpret_cast<uint4*>(q) = make_uint4(pack2(b[0], b[1]), pack2(b[2], b[3]), pack2(b[4], b[5]), pack2(b[6], b[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < live) q[k] = (uint16_t)b[k];
  }
}

// ------------------------------------------------------------------ kernels

struct StepArgs {
  AdamwTable T;
  int64_t lo, hi;          // this launch's tensors
  bool last;               // the last launch of the step
  bool clip;               // factor, and whether the step is taken, from T.control
  float factor;            // otherwise
  float lr_scale;
  const float* lr_factor;  // device, or nullptr
  double beta1, beta2, log1, log2;   // and their logarithms
  float eps;
  uint32_t seed;
  int32_t* step;
  void *m, *v;             // float32, or codes
  float *m_scale, *v_scale;
};

__device__ __forceinline__ bool whole(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether this is the last workgroup of the launch to come here (asked once, by
// one thread); the counter is ready for the next.  No fence: what the others leave
// for the last goes through atomics that have been performed by then.  (A fence of
// device scope writes a whole L2 back, in every workgroup.)
__device__ __forceinline__ bool came_last(uint32_t* counter) {
  auto last_of = [](uint32_t* word, uint32_t all) {
    const bool last = __hip_atomic_fetch_add(word, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == all - 1;
    if (last) __hip_atomic_store(word, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return last;
  };
  const uint32_t parts = min(gridDim.x, (uint32_t)ADAMW_PARTS), part = blockIdx.x % parts;
  return last_of(counter + (part + 1) * ADAMW_LINE, (gridDim.x - part + parts - 1) / parts) && last_of(counter, parts);
}

__device__ __forceinline__ double wave_sum(double s) {
  for (int o = 32; o; o >>= 1) s += shfl_d(s, (int)(threadIdx.x & 63) ^ o);
  return s;
}

// Sums of squares, a workgroup each; the last of the last launch joins them.
__global__ __launch_bounds__(THREADS) void adamw_norm_kernel(AdamwTable T, int64_t lo, int64_t hi, int launch, bool last,
                                                             double grad_scale, double max_norm, float* norm,
                                                             GradList G) {
  __shared__ double part[THREADS / 64];
  __shared__ bool mine;
  // a run of units each, tensor by tensor, four units' loads together
  const int64_t u0 = T.first[lo], all = T.first[hi] - u0, run = (all + gridDim.x - 1) / gridDim.x;
  int64_t u = u0 + run * blockIdx.x;
  const int64_t u1 = min(u + run, u0 + all);
  double s = 0.0;
  while (u < u1) {
    const int k = __builtin_amdgcn_readfirstlane(T.owner[u]);
    const AdamwTensor A = T.tensors[k];
    const void* g = G.p[k - lo];
    const int64_t f = T.first[k], end = min(u1, T.first[k + 1]);
    auto square = [&](const float* v) {
#pragma unroll
      for (int q = 0; q < PER; ++q) s = fma((double)v[q], (double)v[q], s);
    };
    auto four = [&](int dtype) {
      float v[4][PER];
#pragma unroll
      for (int j = 0; j < 4; ++j) load8<true>(g, (u + j - f) * UNIT + threadIdx.x * PER, dtype, PER, v[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) square(v[j]);
    };
    if (whole(g))
      for (; u + 4 <= end && (u + 4 - f) * UNIT <= A.count; u += 4) {
        if (A.dtype == DT_F32) four(DT_F32);
        else if (A.dtype == DT_BF16) four(DT_BF16);
        else four(DT_F16);
      }
    for (; u < end; ++u) {
      const int64_t at = (u - f) * UNIT + threadIdx.x * PER;
      const int live = (int)max((int64_t)0, min((int64_t)PER, A.count - at));
      float v[PER];
      if (live == PER && whole(g)) load8<true>(g, at, A.dtype, live, v);
      else load8<false>(g, at, A.dtype, live, v);
      square(v);
    }
    u = end;
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    // (an exchange: its answer says that it has been performed)
    const uint64_t was = __hip_atomic_exchange(
        reinterpret_cast<uint64_t*>(T.partial) + (int64_t)launch * ADAMW_NORM_GROUPS + blockIdx.x,
        __builtin_bit_cast(uint64_t, (part[0] + part[1]) + (part[2] + part[3])), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::"v"((uint32_t)was), "v"((uint32_t)(was >> 32)) : "memory");
    mine = came_last(T.control + CTL_NORM_COUNT) && last;
  }
  __syncthreads();
  if (!mine) return;
  // (every launch of the norm has as many workgroups)
  s = 0.0;
  for (int64_t k = threadIdx.x; k < (int64_t)(launch + 1) * gridDim.x; k += THREADS)
    s += __hip_atomic_load(T.partial + k / gridDim.x * ADAMW_NORM_GROUPS + k % gridDim.x, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    const double n = sqrt((part[0] + part[1]) + (part[2] + part[3])) * fabs(grad_scale);
    const bool finite = (float)n <= 3.40282347e38f;   // (as the caller sees it)
    T.control[CTL_FACTOR] = __float_as_uint((float)(grad_scale * (n > max_norm ? max_norm / n : 1.0)));
    T.control[CTL_SKIP] = !finite;
    if (norm) *norm = (float)n;
  }
}

// What every element of a step takes.
struct Common {
  float factor, lrf, c1, c2;
  uint32_t key;
  bool skip;
};
__device__ __forceinline__ Common common(const StepArgs& A) {
  Common C;
  C.skip = A.clip && A.T.control[CTL_SKIP] != 0;
  C.factor = A.clip ? __uint_as_float(A.T.control[CTL_FACTOR]) : A.factor;
  C.lrf = A.lr_factor ? A.lr_scale * *A.lr_factor : A.lr_scale;
  const int t = *A.step + 1;
  C.c1 = (float)(-1.0 / expm1((double)t * A.log1));   // (beta 0: the logarithm is -inf, and c 1)
  C.c2 = (float)sqrt(-1.0 / expm1((double)t * A.log2));
  C.key = mix(mix(A.seed) ^ (uint32_t)t);
  return C;
}
// rate: -lr c1.  (v_rcp_f32 is within a step of float32.)
__device__ __forceinline__ float stepped(float p, float m, float r, float rate, float decay, float eps, float c2) {
  return fmaf(rate * m, __builtin_amdgcn_rcpf(fmaf(r, c2, eps)), fmaf(-decay, p, p));
}

// A unit of a tensor: elements `at` on of this thread, `place` in the moments.  FULL: there
// are eight of them, and addresses are aligned.
template <bool SMALL, int DTYPE, bool FULL>
__device__ __forceinline__ void step_unit(const StepArgs& A, const Common& C, const CodeTables* T, const AdamwTensor& P,
                                          const void* grad, int64_t at, int64_t place, int live) {
  const float lr = P.lr * C.lrf, decay = lr * P.weight_decay, rate = -lr * C.c1;
  float g[PER], p[PER];
  uint32_t h[PER];
  load8<FULL>(grad, at, DTYPE, live, g);
  load8<FULL>(P.param, at, DTYPE, live, p);
  const uint32_t key = mix(C.key + (uint32_t)(place >> 32));
#pragma unroll
  for (int q = 0; q < PER; ++q) h[q] = SMALL || DTYPE != DT_F32 ? mix((uint32_t)(place + q) ^ key) : 0u;
  if constexpr (SMALL) {
    // 32 lanes have a block; the ones behind the tensor's last block read the first
    const bool in = FULL || at < (P.count + ADAMW_BLOCK - 1) / ADAMW_BLOCK * ADAMW_BLOCK;
    const int64_t here = in ? place : P.at;
    uint8_t* mc = static_cast<uint8_t*>(A.m) + here;
    uint8_t* rc = static_cast<uint8_t*>(A.v) + here;
    const uint2 mw = *reinterpret_cast<const uint2*>(mc), rw = *reinterpret_cast<const uint2*>(rc);
    const double ms = (double)A.m_scale[here / ADAMW_BLOCK], rs = (double)A.v_scale[here / ADAMW_BLOCK];
    double m[PER], v[PER], mt = 0.0, vt = 0.0;
    bool odd = false;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
#pragma clang fp contract(off)
      const uint32_t cm = (q < 4 ? mw.x : mw.y) >> (8 * (q & 3)) & 255u, cr = (q < 4 ? rw.x : rw.y) >> (8 * (q & 3)) & 255u;
      const double gd = FULL || q < live ? (double)g[q] * (double)C.factor : 0.0;
      const double old = T->m[cm] * ms, root = T->r[cr] * rs;
      m[q] = A.beta1 * old + (1.0 - A.beta1) * gd;
      v[q] = A.beta2 * (root * root) + (1.0 - A.beta2) * gd * gd;
      mt = fmax(mt, fabs(m[q]));
      vt = fmax(vt, v[q]);
      odd |= !(v[q] <= 1.7976931348623157e308);   // (m is finite where v is)
      p[q] = stepped(p[q], (float)m[q], __builtin_amdgcn_sqrtf((float)v[q]), rate, decay, A.eps, C.c2);
    }
    // a block's scales, by their bits: NaN over everything
    uint32_t mb = __float_as_uint((float)(mt / top_value<3>())), rb = __float_as_uint((float)(sqrt(vt) / top_value<4>()));
    if (odd) mb = rb = 0x7fc00000u;
    auto join = [&](uint32_t b) {
      b = max(b, (uint32_t)dpp_i<DPP_XOR1>((int)b));
      b = max(b, (uint32_t)dpp_i<DPP_XOR2>((int)b));
      b = max(b, (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)b));
      b = max(b, (uint32_t)dpp_i<DPP_MIRROR>((int)b));
      return max(b, (uint32_t)shfl_xor_i((int)b, 16));
    };
    mb = join(mb);
    rb = join(rb);
    const double rd = (double)__uint_as_float(rb);
    const double mi = mb ? 1.0 / (double)__uint_as_float(mb) : 0.0, ri = rb ? 1.0 / (rd * rd) : 0.0;
    uint32_t mo[2] = {0, 0}, ro[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      uint32_t cm = code_of_mean(fabs(m[q]) * mi, h[q] & 0xffffu);
      if (cm && m[q] < 0.0) cm |= 128u;
      uint32_t cr = code_of_root(v[q] * ri, h[q] >> 16);
      if (v[q] > 0.0) cr = max(cr, 1u);
      mo[q >> 2] |= cm << (8 * (q & 3));
      ro[q >> 2] |= cr << (8 * (q & 3));
    }
    if (in) {
      *reinterpret_cast<uint2*>(mc) = make_uint2(mo[0], mo[1]);
      *reinterpret_cast<uint2*>(rc) = make_uint2(ro[0], ro[1]);
      if ((threadIdx.x & 31) == 0) {
        A.m_scale[here / ADAMW_BLOCK] = __uint_as_float(mb);
        A.v_scale[here / ADAMW_BLOCK] = __uint_as_float(rb);
      }
    }
  } else {
    float* mp = static_cast<float*>(A.m);
    float* vp = static_cast<float*>(A.v);
    const float b1 = (float)A.beta1, b2 = (float)A.beta2, d1 = (float)(1.0 - A.beta1), d2 = (float)(1.0 - A.beta2);
    float m[PER], v[PER];
    load8<FULL>(mp, place, DT_F32, live, m);
    load8<FULL>(vp, place, DT_F32, live, v);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const float gs = g[q] * C.factor;
      m[q] = fmaf(b1, m[q], d1 * gs);
      v[q] = fmaf(b2, v[q], d2 * gs * gs);
      p[q] = stepped(p[q], m[q], __builtin_amdgcn_sqrtf(v[q]), rate, decay, A.eps, C.c2);
    }
    store8<FULL>(mp, place, DT_F32, live, m, nullptr);
    store8<FULL>(vp, place, DT_F32, live, v, nullptr);
  }
#pragma unroll
  for (int q = 0; q < PER; ++q) h[q] = DTYPE != DT_F32 ? mix(h[q] ^ 0x9e3779b9u) : 0u;
  store8<FULL>(P.param, at, DTYPE, live, p, h);
}

template <bool SMALL>
__global__ __launch_bounds__(THREADS) void adamw_step_kernel(StepArgs A, GradList G) {
  __shared__ Common shared;
  __shared__ std::conditional_t<SMALL, CodeTables, int> tables;
  const CodeTables* T = nullptr;
  if constexpr (SMALL) {
    fill_tables(tables);
    T = &tables;
  }
  if (threadIdx.x == 0) shared = common(A);
  __syncthreads();
  const Common C = shared;
  const int64_t u1 = C.skip ? 0 : A.T.first[A.hi];
  for (int64_t u = A.T.first[A.lo] + blockIdx.x; u < u1; u += gridDim.x) {
    const int k = __builtin_amdgcn_readfirstlane(A.T.owner[u]);
    const AdamwTensor P = A.T.tensors[k];
    const void* grad = G.p[k - A.lo];
    const int64_t start = (u - A.T.first[k]) * UNIT, at = start + threadIdx.x * PER;
    const int live = (int)max((int64_t)0, min((int64_t)PER, P.count - at));
    const int64_t place = P.at + at;   // in the moments, whose last block is whole
    const bool full = start + UNIT <= P.count && whole(grad) && whole(P.param);
    auto go = [&](auto dtype) {
      if (full) step_unit<SMALL, dtype.value, true>(A, C, T, P, grad, at, place, PER);
      else step_unit<SMALL, dtype.value, false>(A, C, T, P, grad, at, place, live);
    };
    if (P.dtype == DT_F32) go(std::integral_constant<int, DT_F32>{});
    else if (P.dtype == DT_BF16) go(std::integral_constant<int, DT_BF16>{});
    else go(std::integral_constant<int, DT_F16>{});
  }
  __syncthreads();
  if (threadIdx.x == 0 && came_last(A.T.control + CTL_STEP_COUNT) && A.last && !C.skip) *A.step += 1;
}

// What 8-bit moments stand for.
__global__ __launch_bounds__(THREADS) void adamw_moments_kernel(const uint8_t* __restrict__ mc, const uint8_t* __restrict__ rc,
                                                                const float* __restrict__ m_scale,
                                                                const float* __restrict__ v_scale, int64_t count,
                                                                float* __restrict__ m, float* __restrict__ v) {
  for (int64_t i = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * 4; i < count; i += (int64_t)gridDim.x * THREADS * 4) {
    const uint32_t mw = *reinterpret_cast<const uint32_t*>(mc + i), rw = *reinterpret_cast<const uint32_t*>(rc + i);
    const double ms = (double)m_scale[i / ADAMW_BLOCK], rs = (double)v_scale[i / ADAMW_BLOCK];
    float mo[4], vo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t cm = mw >> (8 * q) & 255u;
      const double a = code_value<3>(cm & 127u) * ms, r = code_value<4>(rw >> (8 * q) & 255u) * rs;
      mo[q] = (float)(cm & 128u ? -a : a);
      vo[q] = (float)(r * r);
    }
    *reinterpret_cast<float4*>(m + i) = make_float4(mo[0], mo[1], mo[2], mo[3]);
    *reinterpret_cast<float4*>(v + i) = make_float4(vo[0], vo[1], vo[2], vo[3]);
  }
}

}  // namespace

int64_t adamw_units(int64_t count) { return (count + UNIT - 1) / UNIT; }

hipError_t launch_adamw(const AdamwCall& A, hipStream_t st) {
  const AdamwTable& T = A.table;
  // eight workgroups a CU; the norm's launches all have as many, for their join
  const unsigned groups = (unsigned)std::max<int64_t>(1, std::min<int64_t>(T.units, 2048));
  const unsigned norm_groups = std::min<unsigned>(groups, ADAMW_NORM_GROUPS);
  const int64_t launches = std::max<int64_t>(1, (T.count + ADAMW_LAUNCH - 1) / ADAMW_LAUNCH);
  GradList G;
  auto take = [&](int64_t l, int64_t* lo, int64_t* hi) {
    *lo = l * ADAMW_LAUNCH;
    *hi = std::min(T.count, *lo + ADAMW_LAUNCH);
    for (int64_t k = 0; k < ADAMW_LAUNCH; ++k) G.p[k] = *lo + k < *hi ? A.grads[*lo + k] : nullptr;
  };
  hipError_t e;
  if (A.clip)
    for (int64_t l = 0; l < launches; ++l) {
      int64_t lo, hi;
      take(l, &lo, &hi);
      hipLaunchKernelGGL(adamw_norm_kernel, dim3(norm_groups), dim3(THREADS), 0, st, T, lo, hi, (int)l, l + 1 == launches,
                         A.grad_scale, A.max_norm, A.norm, G);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  StepArgs S;
  S.T = T;
  S.clip = A.clip;
  S.factor = (float)A.grad_scale;
  S.lr_scale = A.lr_scale;
  S.lr_factor = A.lr_factor;
  S.beta1 = A.beta1;
  S.beta2 = A.beta2;
  S.log1 = log(A.beta1);
  S.log2 = log(A.beta2);
  S.eps = A.eps;
  S.seed = A.seed;
  S.step = A.step;
  S.m = A.m;
  S.v = A.v;
  S.m_scale = A.m_scale;
  S.v_scale = A.v_scale;
  for (int64_t l = 0; l < launches; ++l) {
    take(l, &S.lo, &S.hi);
    S.last = l + 1 == launches;
    if (A.small)
      hipLaunchKernelGGL(adamw_step_kernel<true>, dim3(groups), dim3(THREADS), 0, st, S, G);
    else
      hipLaunchKernelGGL(adamw_step_kernel<false>, dim3(groups), dim3(THREADS), 0, st, S, G);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_scale, const float* v_scale, int64_t count,
                                float* m_out, float* v_out, hipStream_t st) {
  if (count == 0) return hipSuccess;
  hipLaunchKernelGGL(adamw_moments_kernel, dim3((unsigned)std::min<int64_t>((count / 4 + THREADS - 1) / THREADS, 4096)),
                     dim3(THREADS), 0, st, m, v, m_scale, v_scale, count, m_out, v_out);
  return hipGetLastError();
}

}  // namespace mpq
