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
__device__ __forceinline__ float value_of(uint32_t scale) { return __uint_as_float(scale << 23); }

// Two values over a scale to 8 bits, in the low (HIGH: high) half of w; what is not
// finite becomes NaN. The division is exact, so this is one rounding.
typedef __attribute__((ext_vector_type(2))) short short2v;
template <bool HIGH>
__device__ __forceinline__ uint32_t pack2(uint32_t w, float a, float b, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(__builtin_bit_cast(short2v, w), a, b, scale, HIGH));
}
template <bool HIGH>
__device__ __forceinline__ uint32_t pack2_bf16(uint32_t w, uint32_t pair, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(__builtin_bit_cast(short2v, w), __builtin_bit_cast(bf16x2, pair), scale, HIGH));
}

// Eight neighbouring elements of a row as they lie in memory.
template <bool F32>
struct Eight {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ Eight() {}
  __device__ __forceinline__ explicit Eight(const shl::Raw8<F32>& r) {
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) w[i] = r.w[i / 4][i % 4];
  }
  // The largest magnitude bits that count.
  __device__ __forceinline__ uint32_t magnitude() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
      m = max(m, she::magnitude(__uint_as_float(F32 ? w[i] : w[i] << 16)));
      if (!F32) m = max(m, she::magnitude(__uint_as_float(w[i] & 0xffff0000u)));
    }
    return m;
  }
  // All of them over one scale.
  __device__ __forceinline__ uint2 bytes(float scale) const {
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (F32) {
        o[h] = pack2<false>(0, __uint_as_float(w[4 * h]), __uint_as_float(w[4 * h + 1]), scale);
        o[h] = pack2<true>(o[h], __uint_as_float(w[4 * h + 2]), __uint_as_float(w[4 * h + 3]), scale);
      } else {
        o[h] = pack2_bf16<false>(0, w[2 * h], scale);
        o[h] = pack2_bf16<true>(o[h], w[2 * h + 1], scale);
      }
    }
    return uint2{o[0], o[1]};
  }
};

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
