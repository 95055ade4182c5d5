// The AdamW step's plan and call (adamw.hip, api_tune.hip).
#pragma once
#include <algorithm>
#include "internal.h"

namespace mpq {

constexpr int ADAMW_BLOCK = 256;         // 8-bit moments: elements that share a scale
constexpr int ADAMW_LAUNCH = 440;        // tensors a launch takes (their gradients' addresses are its arguments: 4 KB)
constexpr int ADAMW_NORM_GROUPS = 1024;  // workgroups of the norm's kernel

// Words of the plan's control block.
enum AdamwControl : int { CTL_NORM_COUNT = 0, CTL_STEP_COUNT = 1, CTL_FACTOR = 2, CTL_SKIP = 3, CTL_WORDS = 64 };

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
