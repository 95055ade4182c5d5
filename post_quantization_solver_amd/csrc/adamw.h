// The AdamW step's plan and call (adamw.hip, api_tune.hip).
#pragma once
#include <algorithm>
#include "internal.h"

namespace mpq {

constexpr int ADAMW_BLOCK = 256;         // 8-bit moments: elements that share a scale
constexpr int ADAMW_LAUNCH = 440;        // tensors a launch takes (their gradients' addresses are its arguments: 4 KB)
constexpr int ADAMW_NORM_GROUPS = 1024;  // workgroups of the norm's kernel

// Words of the plan's control block.  A counter has 32 parts and their sum, a cache line
// each: a thousand workgroups that count in one word wait for each other, 10 ns a turn.
constexpr int ADAMW_PARTS = 32, ADAMW_LINE = 32, ADAMW_COUNTER = (ADAMW_PARTS + 1) * ADAMW_LINE;
enum AdamwControl : int {
  CTL_NORM_COUNT = 0,
  CTL_STEP_COUNT = ADAMW_COUNTER,
  CTL_FACTOR = 2 * ADAMW_COUNTER,
  CTL_SKIP,
  CTL_WORDS = 2 * ADAMW_COUNTER + ADAMW_LINE
};

struct AdamwTensor {
  void* param;
  int64_t count, at;
  float lr, weight_decay;
  int32_t dtype, pad;
};
// The plan in device memory.
struct AdamwTable {
  uint32_t* control;
  double* partial;            // launches x ADAMW_NORM_GROUPS
  const AdamwTensor* tensors;
  const int64_t* first;       // count + 1: units before each tensor
  const int32_t* owner;       // units: the tensor of each
  int64_t count, units;
};
struct AdamwCall {
  AdamwTable table;
  const void* const* grads;   // host
  bool small, clip;
  double grad_scale, max_norm;
  float lr_scale;
  const float* lr_factor;
  double beta1, beta2;
  float eps;
  uint32_t seed;
  int32_t* step;
  void *m, *v;
  float *m_scale, *v_scale;
  float* norm;
};
int64_t adamw_units(int64_t count);
hipError_t launch_adamw(const AdamwCall& A, hipStream_t st);
hipError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_scale, const float* v_scale, int64_t count,
                                float* m_out, float* v_out, hipStream_t st);

}  // namespace mpq
