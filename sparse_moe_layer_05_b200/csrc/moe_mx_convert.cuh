// moe_mx_convert.cuh -- the scale rule of the OCP Microscaling conversion,
// shared by the kernels that write MX blocks (activations of the quantised
// modes, the norm's 8-bit checkpoint).
#pragma once

#include <stdint.h>

#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// Exponent of the shared scale X = 2^(floor(log2 max|v|) - emax), emax 8 for
// E4M3 and 2 for E2M1, kept in the E8M0 range (at least -127: groups whose
// max|v| is below 2^(emax - 127) keep that smallest scale); an all-zero group
// takes X = 1.
template <int ACT>
__device__ __forceinline__ int mx_scale_exp(float amax) {
  constexpr int emax = ACT == ACT_E2M1 ? 2 : 8;
  if (!(amax > 0.f)) return 0;
  const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 127;  // floor(log2)
  return max(e - emax, -127);
}

// E8M0 byte -> 2^(s - 127) (byte 0 is the fp32 subnormal 2^-127; 255 is NaN).
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}

// The same for a checkpointed row whose inverse root is r: 0 where r is, so that the
// row is zeros. A row that held an infinity has r = 0 and codes for 1.75 2^128, which
// is fp32's infinity, and that times r would be a NaN.
__device__ __forceinline__ float e8m0_of_row(uint32_t s, float r) {
  return r == 0.f ? 0.f : e8m0_to_f32(s);
}

}  // namespace moe
