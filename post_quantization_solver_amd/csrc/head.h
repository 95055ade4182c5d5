// A head's cross entropy and its gradients (head.hip, api_tune.hip).
#pragma once
#include "qlayer.h"

namespace mpq {

struct HeadArgs {
  QLayer L;                            // the head (a matrix: its m and n alone)
  const void* W; int64_t ldw;          // a matrix of x's type, or nullptr
  const void* x; int64_t ldx;
  int dtype;
  int64_t t;
  const float* bias;                   // per row of the head
  const int32_t* targets;
  const float* weights;                // per token (nullptr: 1)
  float* loss;
  bool dense, need_dx, need_dhead;
  void* dx; int64_t lddx;
  float *dscale, *doffset, *dbias;     // dscale, doffset: of a packed head
  void* dW; int64_t lddw;              // of a matrix
};
constexpr float H_LOG2E = 1.44269504f;

// A piece of the vocabulary: some rows of the head, all tokens.
struct PieceArgs {
  const float* S; int64_t lds;     // t x m: s, where it is in memory
  int64_t t, m, row0;              // the piece's tokens and rows, the first of them
  const float *a, *o, *b;          // of the piece's rows (nullptr: 1, 0, 0)
  const float* levels; int mid;    // s is of entries less levels[mid] (mid < 0: as they are)
  int centre;                      // as mid, of the entries that dz meets
  const float *weight, *sum;
  const int32_t* targets;
  float* target_z;
  float2* part;                    // per segment and token: the largest, the sum
  // gradients
  const float *row_top, *row_scale, *row_target;   // the largest, w / sum of exponentials, dz of the target
  const uint32_t* tmax;            // the bounds that dz^T's rows are scaled by
  const float* fmax;               // the largest factor of dz, in 64 parts (nullptr: 1)
  const uint32_t* xmax;            // the tokens' factors in x's operand: dz^T carries the inverse
  const uint32_t* refs;            // the weights' planes' factors (nullptr: a is dz's factor)
  uint32_t* dmax;                  // the bound that a token's d is scaled by
  uint16_t* d; int64_t plane_d, mp; int terms_d;    // dz times its factors: t rows of mp (nullptr: none)
  bool raw_d;                      // dz itself, in bfloat16
  bool own_target;                 // the targets' left out
  float* rowpart;                  // t x (mp / 64): sums of dz o' (nullptr: none)
  uint16_t* dt; int64_t plane_t, tp; int terms_t;   // dz^T: m rows of tp (nullptr: none)
  float* colpart;                  // (tp / 64) x 3 x m: sums of dz, dz s, dz X (nullptr: none)
  float *dbias, *dscale, *doffset; // or those themselves, where there is one tile of tokens
};

#ifdef __HIPCC__
// Four float16 terms of v at p[0 .. 3].
__device__ __forceinline__ void put_terms(uint16_t* p, int64_t plane, int planes, const float* v) {
  uint32_t b[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) f16_terms(v[k], b[k]);
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(b[0][0], b[1][0]), pack2(b[2][0], b[3][0]));
  if (planes > 1)
    *reinterpret_cast<uint2*>(p + plane) = make_uint2(pack2(b[0][1], b[1][1]), pack2(b[2][1], b[3][1]));
}
// Four values of dz times their factors as d's operand.
__device__ __forceinline__ void put_dz(const PieceArgs& A, int64_t t, int64_t i, const float* u) {
  if (A.raw_d)
    *reinterpret_cast<uint2*>(A.d + q_at(t, i, A.mp)) = make_uint2(OpBf16::pack(u[0], u[1]), OpBf16::pack(u[2], u[3]));
  else
    put_terms(A.d + q_at(t, i, A.mp), A.plane_d, A.terms_d, u);
}
__device__ __forceinline__ float largest_factor(const PieceArgs& A) {
  if (!A.fmax) return 1.f;
  uint32_t top = abs_bits(A.fmax[threadIdx.x & 63]);
  for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)shfl_xor_i((int)top, o));
  return __uint_as_float(top);
}
// Over the sixteen lanes of a row.
__device__ __forceinline__ float sum16(float s) {
  s += dpp_f<DPP_XOR1>(s);
  s += dpp_f<DPP_XOR2>(s);
  s += dpp_f<DPP_HALF_MIRROR>(s);
  s += dpp_f<DPP_MIRROR>(s);
  return s;
}
#endif

// A piece's logits straight from the product's registers (headgemm.hip): the statistics
// (grads = false) or dz and its sums.  Tiles of head_tile() rows by columns: part has a
// segment per tile of rows, rowpart a column each, colpart a row per tile of tokens.
struct HeadTile {
  int rows, tokens;
};
HeadTile head_tile(int64_t m, int64_t t);
hipError_t launch_head_gemm(const QGemm& g, const PieceArgs& A, const uint32_t* rowmax, bool grads, hipStream_t st);

// dx's sums over the pieces, `splits` of t x ldo (a piece has `rows` rows, the last may
// have fewer): added to, but for the first piece.  g: the planes of the head with their
// rows as depth (g.arows of them), dz.
int head_dx_splits(int64_t n, int64_t t, int64_t rows, int npairs);
hipError_t launch_head_dx(const QGemm& g, const uint32_t* rowmax, float* out, int64_t ldo, int64_t rows, bool first,
                          hipStream_t st);

size_t head_workspace(const HeadArgs& A);
hipError_t launch_head(const HeadArgs& A, void* ws, hipStream_t st);

}  // namespace mpq
