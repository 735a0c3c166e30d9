// Device helpers of the operators around the share (norms, 8-bit products, the
// share for a few tokens).
#pragma once

#include "moe_device.h"

namespace moe {

// f32_to_bf16_bits' rounding by the conversion instruction, for values that may be
// infinite or NaN (a NaN stays one).
__device__ __forceinline__ uint16_t cvt_bf16(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  return uint32_t(cvt_bf16(lo)) | (uint32_t(cvt_bf16(hi)) << 16);
}

// Sum over the wave as in wave_max_dpp (no LDS traffic), the same on every lane.
__device__ __forceinline__ float wave_sum_dpp(float v) {
  auto step = [](float x, auto ctrl) {
    constexpr int c = decltype(ctrl)::value;
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), c, 0xF, 0xF, false));
  };
  v = step(v, std::integral_constant<int, 0xB1>{});
  v = step(v, std::integral_constant<int, 0x4E>{});
  v = step(v, std::integral_constant<int, 0x141>{});
  v = step(v, std::integral_constant<int, 0x140>{});
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace moe
