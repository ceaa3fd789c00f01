// Shared by the kernels of linear attention with a decay for each head.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace sla {

#ifdef __CUDACC__
// decay^n = 2^(n l2), l2 = log2 of the head's decay (-inf for a decay of
// zero).  The product's rounding is 2^-24 of the exponent: a weight that
// matters (2^-20 and up) is off by at most 20 * 2^-24 * ln 2, under 2^-20.
__device__ __forceinline__ float decay_log2(float log_decay) { return log_decay * 1.4426950408889634f; }
__device__ __forceinline__ float decay_power(float l2, int n) {
  return n == 0 ? 1.f : exp2f(static_cast<float>(n) * l2);
}

// Real tokens of sequence b, and of its segment `seg`.
__device__ __forceinline__ int sequence_tokens(const DecayPlan& P, const int32_t* lens, int b) {
  return lens ? min(max(lens[b], 0), P.N) : P.N;
}
__device__ __forceinline__ int segment_tokens(const DecayPlan& P, const int32_t* lens, int b, int seg) {
  return min(max(sequence_tokens(P, lens, b) - seg * P.seg_len, 0), P.seg_len);
}
#endif

}  // namespace sla
