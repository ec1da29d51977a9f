// Device code shared by the experts' kernels: the 8-bit format.
#pragma once

#include "experts_kernels.h"
#include "layer_device.h"

namespace she {

typedef __attribute__((ext_vector_type(4))) int int4v;
typedef __attribute__((ext_vector_type(8))) int int8v;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// Magnitude bits that count for a scale: none of what is not finite.
__device__ __forceinline__ uint32_t magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u > 0x7f7fffffu ? 0u : u;
}
// The scale's biased exponent: 448 = 1.75 * 2^8, so a magnitude 1.f * 2^x takes x - 8,
// and one more where 1.f is over 1.75.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(max(e, 1));
}
__device__ __forceinline__ float inverse_of(uint32_t scale) { return __uint_as_float((254u - scale) << 23); }
__device__ __forceinline__ float value_of(uint32_t scale) { return __uint_as_float(scale << 23); }

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// Four bytes in 8 bits times a scale, exactly.
__device__ __forceinline__ void widen(int w, float scale, bf16x8& out, int at) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
  out[at] = a[0];
  out[at + 1] = a[1];
  out[at + 2] = b[0];
  out[at + 3] = b[1];
}

// Offset e of the experts' rows, within the batch whatever it holds.
__device__ __forceinline__ int group_row(const Groups& g, int e) { return min(max(g.offsets[e], 0), g.n); }

}  // namespace she
