// What happens to finished sums of the feed-forward block's products, eight
// columns of one row at a time (layer_gemm.hip, layer_decode.hip).
#pragma once

#include "layer_device.h"
#include "layer_kernels.h"

namespace shl {

// ---------------------------------------------------------------- activation
// Value a and derivative da at g. SiLU is g s(g), s the logistic function; the
// tanh form of GELU is g s(t), t = 2 k (g + c g^3), k = sqrt(2 / pi), c =
// 0.044715, since (1 + tanh(x)) / 2 = s(2 x). So both are g s(g (p + q g^2)).
struct Activation {
  float p, q;
  bool relu;
  __device__ __forceinline__ explicit Activation(int act) {
    const float k2 = 1.5957691216057308f;
    p = act == kGelu ? k2 : 1.f;
    q = act == kGelu ? k2 * 0.044715f : 0.f;
    relu = act == kRelu;
  }
  __device__ __forceinline__ void operator()(float g, float& a, float& da) const {
    const float g2 = fminf(g * g, 1e30f);  // q g^2 stays a number where q = 0
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-g * (p + q * g2)));
    a = g * s;
    da = s + a * (1.f - s) * (p + 3.f * q * g2);
    if (relu) {
      a = g > 0.f ? g : g != g ? g : 0.f;
      da = g > 0.f ? 1.f : 0.f;
    }
  }
};

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.f;
}

// Raises a maximum word by a wave's largest finite |value|. The order of the
// atomics does not change the result. They queue up at a word, so that every
// workgroup has one of kMaxParts (1024 on one word: 42 us for a finish kernel
// that now takes 12), and it does not look at the word first (16 us).
__device__ __forceinline__ void raise_max(uint32_t* word, float m) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const uint32_t bits = __float_as_uint(m);
  if ((threadIdx.x & 63) == 0 && bits) atomicMax(word, bits);
}

// Power of two that an operand's planes are scaled by: its largest finite
// |value| comes into [2^14, 2^15).
__device__ __forceinline__ int scale_exp(uint32_t word) {
  if (word == 0) return 0;
  const int e = static_cast<int>(word >> 23);
  return 14 - ((e ? e : 1) - 127);
}

// The epilogue on columns [col, col + 8) of one row: v (and for kGate also w,
// the same columns of u; for kActBwd g and u as they lie in memory). oc, og: the
// place in the results and in g and u. Columns from N to pad_to get zeros.
// Returns the largest finite |value| of a result that a later product reads.
// bf16 g and u are rounded where they are kept (the activation takes them before
// that): the kept state and this epilogue's traffic, which is as long as its
// product at ordinary widths, would double without.
template <bool F32, int EPI>
__device__ __forceinline__ float finish8(const EpiArgs& e, const Activation& act, int problem, int64_t oc, int64_t og, int col, int N,
                                         float (&v)[8], float (&w)[8], const Raw8<F32>& gr, const Raw8<F32>& ur) {
  const int width = e.pad_to > N ? e.pad_to : N;
  // all but a kStore's rows are padded to whole groups of eight
  const int n = EPI == kStore ? min(8, width - col) : col < width ? 8 : 0;
  float m = 0.f;
  if (n <= 0) return m;
  if (col + 8 > N) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i >= N) v[i] = 0.f, w[i] = 0.f;
  }
  if (EPI == kStore) {
    store8(problem ? e.c[1] : e.c[0], oc, n, F32, v);
  } else if (EPI == kGate) {
    if (e.g) {
      store8(e.g, og, 8, F32, v);
      store8(e.u, og, 8, F32, w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      act(v[i], a, da);
      v[i] = a * w[i];
      if (F32) m = fmaxf(m, finite_abs(v[i]));
    }
    store8(e.c[0], oc, 8, F32, v);
  } else {
    float g[8], u[8];
    unpack8<F32>(gr, g);
    unpack8<F32>(ur, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      act(g[i], a, da);
      g[i] = v[i] * u[i] * da;
      u[i] = v[i] * a;
      if (F32) m = fmaxf(m, fmaxf(finite_abs(g[i]), finite_abs(u[i])));
    }
    store8(e.c[0], oc, 8, F32, g);
    store8(e.c[1], oc, 8, F32, u);
  }
  return m;
}

// What kActBwd reads of g and u for eight columns of a row.
template <bool F32>
__device__ __forceinline__ void load_gu(const EpiArgs& e, bool row_in, int64_t og, int col, int N, Raw8<F32>& g, Raw8<F32>& u) {
  const int width = e.pad_to > N ? e.pad_to : N;
  if (row_in && col < width) {
    g = load_raw8<F32>(e.g, og, 0, 8);
    u = load_raw8<F32>(e.u, og, 0, 8);
  }
}

}  // namespace shl
