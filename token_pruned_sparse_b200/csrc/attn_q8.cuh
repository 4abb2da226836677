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

// A key scale of 0 (an empty block) stands for logits of 0: the smallest positive factor gives just that.
constexpr float kFactorMin = 1.17549435e-38f;
constexpr float kScaleMin = 7.8886091e-31f, kScaleMax = 1.2676506e30f;   // 2^-100, 2^100

// A row has two references (log2): m, the largest x + log2 vs less a raise r, which P' and O count in, and s, the
// largest x, which the sum l counts in (the largest when they were set). The largest P' is then 2^r or more and f16's
// subnormals end at 2^-(25 + r) of it, so a range of n keys loses n 2^-(25 + r) of its largest term at most (with
// r = 0, 3% at a million keys). A high r leaves less room for the keys to come: rows meet a new reference sooner.
// So r grows with the range (raise_of): n 2^-(25 + r) <= 2^-13 up to 2^20 keys, and 2^-33 of them beyond. r = 8
// everywhere takes 428 us instead of 385 for a masked call of 24 blocks a row, where r = 0 does, and 725 instead of
// 714 for 6,084 rows over 20,280 keys (r = 3), on one GPU. The few-row kernel's references cost little: r = kRaise.
// A key's share of the sum is P' 2^(m - log2 vs - s). Up to kShareMax of that factor a P' that underflows (2^-126) is
// of a key below 2^-66 of the sum. Beyond it (blocks whose vs is far below others'), and where vs is 0 (values of 0:
// P' = 0), a pass of exponentials of its own takes the sum: with a quarter of the blocks empty 6,084 rows over 20,280
// keys take 748 us instead of 614 (empty tiles on the fast path instead spilled registers, 739 us for every call).
constexpr int kRaise = 8;
__device__ __forceinline__ float raise_of(int tiles) {   // of 128 keys: ceil(log2(tiles)) - 5, from 0 to kRaise
  const int r = 27 - __clz(tiles - 1);
  return static_cast<float>(r < 0 ? 0 : (r > kRaise ? kRaise : r));
}
constexpr float kShareMax = 1.1529215e18f;   // 2^60
__device__ __forceinline__ float share_of(float m, float lv, float s) {
  return fminf(fast_exp2(m - lv - s), 3e38f);   // finite: it may meet sums of 0 (NaN, without references yet: 3e38)
}
// log2 of a V scale; -inf for 0, and for a negative or NaN one, which counts as 0
__device__ __forceinline__ float log2_scale(float vs) {
  return vs > 0.f ? __log2f(fminf(fmaxf(vs, kScaleMin), kScaleMax)) : -INFINITY;
}

// l += y, with what the addition rounds off (of y, which takes in the last such rest) kept in low
__device__ __forceinline__ void add_low(float y, float& l, float& low) {
  const float t = l + y;
  low = y - (t - l);
  l = t;
}

// Weight of a partial sum l_part in units of 2^s_part in one of 2^s: 0 without a key, NaN where the sum is NaN (its
// reference may then be -inf).
__device__ __forceinline__ float part_weight(float s_part, float l_part, float s) {
  if (l_part != l_part) return l_part;
  return s_part == -INFINITY ? 0.f : fast_exp2(s_part - s);
}
// Weight of a partial O in units of 2^m_part against sums in units of 2^s: 0 if it has no key with a value.
__device__ __forceinline__ float value_weight(float m_part, float s) {
  return m_part == -INFINITY ? 0.f : fast_exp2(m_part - s);
}

// At most kFewRows rows of a dense call (attn_q8_few.cu).
constexpr int kFewRows = 16;
constexpr int kFewMaxSplit = 128;
int few_split(int64_t cap, int64_t N, int H);
int launch_attn_q8_few(const Q8Args& prm, cudaStream_t st);

}  // namespace tps
