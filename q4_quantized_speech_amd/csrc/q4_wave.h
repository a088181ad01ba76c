// Reductions over a wave without LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_device.h"

namespace q4 {

// The largest over the wave's lanes (NaN loses), in all of them: DPP within each
// row of 16, then the rows' swaps.
__device__ __forceinline__ float wave64_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The sum over the wave's lanes, the same bits in all of them.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  i32x2 b = __builtin_bit_cast(i32x2, v);
  b.x = __builtin_amdgcn_update_dpp(0, b.x, CTRL, 0xF, 0xF, false);
  b.y = __builtin_amdgcn_update_dpp(0, b.y, CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, b);
}
__device__ __forceinline__ double wave64_sum(double v) {
  typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  u32v2 b = __builtin_bit_cast(u32v2, v);
  auto x = __builtin_amdgcn_permlane16_swap(b.x, b.x, false, false);
  auto y = __builtin_amdgcn_permlane16_swap(b.y, b.y, false, false);
  v = __builtin_bit_cast(double, u32v2{x[0], y[0]}) + __builtin_bit_cast(double, u32v2{x[1], y[1]});
  b = __builtin_bit_cast(u32v2, v);
  x = __builtin_amdgcn_permlane32_swap(b.x, b.x, false, false);
  y = __builtin_amdgcn_permlane32_swap(b.y, b.y, false, false);
  return __builtin_bit_cast(double, u32v2{x[0], y[0]}) + __builtin_bit_cast(double, u32v2{x[1], y[1]});
}

}  // namespace q4
