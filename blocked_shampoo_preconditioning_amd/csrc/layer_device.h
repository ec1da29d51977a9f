// Device code shared by the layer operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace shl {

typedef __attribute__((ext_vector_type(4))) float floatx4;
typedef __attribute__((ext_vector_type(4))) uint32_t uint4v;

__device__ __forceinline__ float bf16_to_f32(uint32_t v) { return __uint_as_float(v << 16); }
// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  return (u & 0x7fffffffu) > 0x7f800000u ? (u >> 16) | 0x40u : r;
}

// Eight consecutive elements of a row, or its last n < 8 (the others 0).
// Whole groups go as 16-byte accesses whatever their alignment (global memory
// takes unaligned ones).
__device__ __forceinline__ void load8(const void* p, int64_t off, int n, bool f32, float (&v)[8]) {
  if (f32) {
    const float* q = static_cast<const float*>(p) + off;
    if (n == 8) {
      floatx4 a, b;
      __builtin_memcpy(&a, q, 16);
      __builtin_memcpy(&b, q + 4, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? q[i] : 0.f;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + off;
    if (n == 8) {
      uint4v w;
      __builtin_memcpy(&w, q, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_to_f32(w[i] & 0xffffu), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(q[i]) : 0.f;
    }
  }
}

__device__ __forceinline__ void store8(void* p, int64_t off, int n, bool f32, const float (&v)[8]) {
  if (f32) {
    float* q = static_cast<float*>(p) + off;
    if (n == 8) {
      floatx4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = v[i], b[i] = v[4 + i];
      __builtin_memcpy(q, &a, 16);
      __builtin_memcpy(q + 4, &b, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = v[i];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + off;
    if (n == 8) {
      uint4v w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(v[2 * i]) | (f32_to_bf16(v[2 * i + 1]) << 16);
      __builtin_memcpy(q, &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = static_cast<uint16_t>(f32_to_bf16(v[i]));
    }
  }
}

}  // namespace shl
