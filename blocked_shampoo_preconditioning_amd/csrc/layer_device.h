// Device code shared by the layer operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace shl {

typedef __attribute__((ext_vector_type(4))) float floatx4;
typedef __attribute__((ext_vector_type(4))) uint32_t uint4v;

__device__ __forceinline__ float bf16_to_f32(uint32_t v) { return __uint_as_float(v << 16); }
// Two fp32 values to bf16, to nearest even (the hardware's conversion; NaN
// stays NaN), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) float f2;
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  const f2 x = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, b2));
}
__device__ __forceinline__ uint16_t f32_to_bf16(float x) { return static_cast<uint16_t>(pack_bf16(x, 0.f)); }

// Eight elements as they lie in memory: held so, a row on its way takes half
// (bf16) or as many registers as its values.
template <bool F32>
struct Raw8 {
  uint4v w[F32 ? 2 : 1];
};

// Elements [col, col + n) of a row that starts at p + row, n <= 8 of them (the
// others 0). Whole groups go as 16-byte accesses whatever their alignment
// (global memory takes unaligned ones). A row's last group n < 8 reads the
// row's last eight, which settle8 moves down, since a loop over single elements
// would wait for each; only rows shorter than eight are read so. Loads that
// are to be in flight together are all fetched before the first is settled.
template <bool F32>
__device__ __forceinline__ Raw8<F32> fetch8(const void* p, int64_t row, int col, int n) {
  constexpr int E = F32 ? 4 : 2, W = F32 ? 8 : 4;
  Raw8<F32> r;
  uint32_t w[W];
  if (n > 0 && (n == 8 || col >= 8)) {
    __builtin_memcpy(w, static_cast<const char*>(p) + (row + col - (8 - n)) * E, 8 * E);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    if (n > 0) {
#pragma unroll 1
      for (int k = n - 1; k >= 0; --k) {
        if constexpr (F32) {
#pragma unroll
          for (int i = 7; i > 0; --i) w[i] = w[i - 1];
          w[0] = static_cast<const uint32_t*>(p)[row + col + k];
        } else {
#pragma unroll
          for (int i = 3; i > 0; --i) w[i] = w[i] << 16 | w[i - 1] >> 16;
          w[0] = w[0] << 16 | static_cast<const uint16_t*>(p)[row + col + k];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) r.w[i / 4][i % 4] = w[i];
  return r;
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> settle8(Raw8<F32> r, int col, int n) {
  constexpr int W = F32 ? 8 : 4;
  const int up = 8 - n;  // elements that were read before col
  if (n > 0 && n < 8 && col >= 8) {
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = r.w[i / 4][i % 4];
#pragma unroll
    for (int b = 4; b > 0; b >>= 1) {
      if (up & b) {
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = i + b < 8 ? w[i + b < 8 ? i + b : 7] : 0u;
        } else if (b == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = w[i] >> 16 | (i < 3 ? w[i < 3 ? i + 1 : 3] << 16 : 0u);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = i + b / 2 < 4 ? w[i + b / 2 < 4 ? i + b / 2 : 3] : 0u;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i / 4][i % 4] = w[i];
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* p, int64_t row, int col, int n) {
  return settle8<F32>(fetch8<F32>(p, row, col, n), col, n);
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (F32)
      v[i] = __uint_as_float(r.w[F32 ? i / 4 : 0][i % 4]);
    else
      v[i] = __uint_as_float(i % 2 ? r.w[0][i / 2] & 0xffff0000u : r.w[0][i / 2] << 16);
  }
}

// Eight elements to a row, or its last n < 8: one by one in a rolled loop over
// a shifting register file, since these lines are in every kernel many times and
// fetching instructions costs more than that loop.
__device__ __forceinline__ void store8(void* p, int64_t off, int n, bool f32, const float (&v)[8]) {
  if (n == 8) {
    if (f32) {
      float* q = static_cast<float*>(p) + off;
      floatx4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = v[i], b[i] = v[4 + i];
      __builtin_memcpy(q, &a, 16);
      __builtin_memcpy(q + 4, &b, 16);
    } else {
      uint4v w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      __builtin_memcpy(static_cast<uint16_t*>(p) + off, &w, 16);
    }
    return;
  }
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v[i];
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    if (f32)
      static_cast<float*>(p)[off + k] = x[0];
    else
      static_cast<uint16_t*>(p)[off + k] = f32_to_bf16(x[0]);
#pragma unroll
    for (int i = 0; i < 7; ++i) x[i] = x[i + 1];
  }
}

}  // namespace shl
