// What the two kernels of pruned_attn_q8 share: the arguments, and the limits of scales.
#pragma once

#include "attn_common.cuh"

namespace tps {

struct Q8Args {
  AttnArgs a;          // a.k = K's codes; a.v is not used
  const uint8_t* v8;
  const float* ks;
  const float* vs;
  float scale_log2;
  int nsplit;          // key ranges
  float* o_part;       // nsplit > 1: normalised fp32 partials [nsplit][part_rows][H][D] and their
  float* lse_part;     // log-sum-exp [nsplit][part_rows][H], of the rows from part_row0
  int64_t part_rows;
  int64_t part_row0;
  int tile0;           // first row tile of this launch
  unsigned int* status;
};

// A scale of 0 (an empty block) stands for values of 0: the smallest positive factors give just that.
constexpr float kFactorMin = 1.17549435e-38f;
constexpr float kScaleMin = 7.8886091e-31f, kScaleMax = 1.2676506e30f;   // 2^-100, 2^100

// Weight of a partial result with maximum m_part (log2) and sum l_part against the maximum m of all: 0 without a
// key, NaN where the sum is NaN (its maximum may then be -inf).
__device__ __forceinline__ float part_weight(float m_part, float l_part, float m) {
  if (l_part != l_part) return l_part;
  return m_part == -INFINITY ? 0.f : fast_exp2(m_part - m);
}

// At most kFewRows rows of a dense call (attn_q8_few.cu).
constexpr int kFewRows = 16;
constexpr int kFewMaxSplit = 128;
int few_split(int64_t cap, int64_t N, int H);
int launch_attn_q8_few(const Q8Args& prm, cudaStream_t st);

}  // namespace tps
