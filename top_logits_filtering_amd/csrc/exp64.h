// exp in 64 bits, and the table of it over bf16 values: plain functions, which the
// host's tests run as well.
#pragma once

#include <stdint.h>

#pragma clang force_cuda_host_device begin

namespace tkp {

// exp(x - ref) in 64 bits, 0 for -inf and NaN: 2^(n + r) with n whole and r in
// [-1/2, 1/2], 2^r by the polynomial of degree 9 that meets it at the Chebyshev
// points, within 1.9e-14 of it. What is added to round to n leaves n in the low bits.
// 16 instructions; the library's exp takes about 30.
__attribute__((always_inline)) inline double exp_from(float x, float ref) {
  constexpr double kLog2e = 1.4426950408889634, kRound = 6755399441055744.0;  // 1.5 * 2^52
  const double d = __builtin_fmax(static_cast<double>(x) - static_cast<double>(ref), -760.0);
  const double t = __builtin_fma(d, kLog2e, kRound);
  const double r = __builtin_fma(d, kLog2e, kRound - t);
  double e = 1.0205905413765595e-07;
  e = __builtin_fma(e, r, 1.325964524488711e-06);
  e = __builtin_fma(e, r, 1.5252672924850737e-05);
  e = __builtin_fma(e, r, 0.0001540343375125101);
  e = __builtin_fma(e, r, 0.0013333558200794592);
  e = __builtin_fma(e, r, 0.009618129193934313);
  e = __builtin_fma(e, r, 0.05550410866465167);
  e = __builtin_fma(e, r, 0.2402265069564034);
  e = __builtin_fma(e, r, 0.6931471805599462);
  e = __builtin_fma(e, r, 1.0000000000000135);
  return __builtin_ldexp(e, static_cast<int>(static_cast<uint32_t>(__builtin_bit_cast(uint64_t, t))));
}

// exp of the bf16 values of sizes from 2^-53 up to 2^7: smaller ones are taken as
// 2^-53, whose entries are 1.0, within 2^-53 of exp; -128 and below as -128, whose
// entry is 0. Larger than 128 there are none.
constexpr int kTableLow = 74 << 7, kTableHigh = 134 << 7;  // bits of 2^-53 and 2^7
constexpr int kTableSign = 8192;                           // entries of the negative ones come behind
constexpr int kTable = kTableSign + kTableHigh - kTableLow + 1;
static_assert(kTableHigh - kTableLow < kTableSign);
constexpr int kTableNear = 118 << 7;  // bits of 2^-9: below, four terms of the series are within 2^-52

// The entry of the values whose size has the bits m, kTableLow <= m <= kTableHigh.
__attribute__((always_inline)) inline void table_pair(int m, double& up, double& down) {
  const float x = __builtin_bit_cast(float, static_cast<uint32_t>(m) << 16);
  if (m == kTableLow) {
    up = down = 1.0;
  } else if (m < kTableNear) {
    const double d = x;
    const double even = __builtin_fma(d * d, __builtin_fma(d * d, 1.0 / 24, 0.5), 1.0);
    const double odd = __builtin_fma(d * d, 1.0 / 6, 1.0) * d;
    up = even + odd;
    down = even - odd;
  } else {
    up = exp_from(x, 0.0f);
    down = m == kTableHigh ? 0.0 : exp_from(-x, 0.0f);
  }
}

}  // namespace tkp

#pragma clang force_cuda_host_device end
