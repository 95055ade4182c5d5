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
size_t head_workspace(const HeadArgs& A);
hipError_t launch_head(const HeadArgs& A, void* ws, hipStream_t st);

}  // namespace mpq
