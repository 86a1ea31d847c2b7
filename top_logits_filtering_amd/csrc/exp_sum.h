// Sums of exp over chunks of a row in 32 bits, with what the argument's rounding
// loses put right: 7 or 8 instructions an element, and a known error.
#pragma once

#include <float.h>

#include "device_common.h"

namespace tkp {

// The chunks' sums are taken of exp(x) itself while the chunk's maximum lies
// in [kLowMax, kHighMax], which a model's logits do: then no maximum is needed
// before the sum. Other chunks are read and summed again in 64 bits, less their
// maximum.
constexpr float kHighMax = 80.0f;  // eight terms of exp(80) stay finite
constexpr float kLowMax = -40.0f;  // terms that exp2 flushes are below 2^-68 of the largest

constexpr float kLn2 = 0.693147180559945309417f;

// exp(x) = 2^t * 2^lo with t as the hardware's exp2 takes it: returns 2^t and
// adds to `rest` what the sum needs for 2^lo (sum_of).
// fp32: t = x log2(e) rounded, lo what that lost; rest is the sum of lo * 2^t.
// 16-bit types, whose values have at most 8 or 11 bits: t = x * log2_high(),
// which has so few that the product is exact; rest is the sum of x * 2^t.
template <class DT>
constexpr float log2_high() {
  return DT::kNegInf == 0xFF80u ? 47274.0f / 32768 : 5909.0f / 4096;
}
template <class DT>
__device__ __forceinline__ float exp_parts(float x, float& rest) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.925963033500e-8f;
  const float xc = __builtin_amdgcn_fmed3f(x, -104.0f, 104.0f);  // finite, also for -inf
  if constexpr (DT::kPerVec == 4) {
    const float t = xc * kLog2e;
    const float lo = __builtin_fmaf(xc, kLog2eLow, __builtin_fmaf(xc, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    rest = __builtin_fmaf(e, lo, rest);
    return e;
  } else {
    const float e = __builtin_amdgcn_exp2f(xc * log2_high<DT>());
    rest = __builtin_fmaf(e, xc, rest);
    return e;
  }
}

// The sum of exp(x) out of the sums of 2^t and rest.
// fp32: 2^lo = 1 + lo ln 2, as lo is below 2^-17.
// 16-bit types: exp(x) = 2^t * exp(kx) with k = 1 - log2_high() ln 2, 4.9e-6 or
// 4.7e-5. With m the mean of x under the weights 2^t the sum is
// sum * exp(km) * (1 + k^2 var / 2 + ...). The variance of 257 elements, as many
// as a thread has, is at most 9 (255 of them lie about 6 below the others), so
// what is left out is below 1e-8; |km| is below 5e-3.
template <class DT>
__device__ __forceinline__ double sum_of(double sum, double rest) {
  if constexpr (DT::kPerVec == 4) return sum + rest * kLn2;
  constexpr double kRate = 1.0 - log2_high<DT>() * 0.693147180559945309417;
  const double y = rest * kRate, z = y * __builtin_amdgcn_rcp(sum + 0x1p-1000);
  return sum + y * (1.0 + z * (0.5 + z * (1.0 / 6)));
}

// Relative error of a chunk's sum: 8.5e-8 of exp2 (the most over all arguments
// from -126 to 126, measured; below them it gives 0), three additions in fp32 at
// 2^-24 each, and either a multiply-add at 2^-24 or the 1e-8 of sum_of; less than
// 1e-10 of what follows in 64 bits.
constexpr double kSumError = 3.5e-7;

// Elements of a row of V before its first 16-byte boundary.
template <class raw_t>
__device__ __forceinline__ int head_of(const raw_t* row, int V) {
  const int bytes = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u);
  const int head = bytes / static_cast<int>(sizeof(raw_t));
  return head < V ? head : V;
}

}  // namespace tkp
