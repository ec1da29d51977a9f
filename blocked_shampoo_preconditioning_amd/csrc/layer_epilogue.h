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
// bf16 takes the hardware's exponential and reciprocal, whose errors (the first's
// grows with its argument: 62 steps of fp32 at -80) its own rounding covers; fp32
// the exact ones, which an epilogue has time for (step of 4096 x 768 x 2048 the same).
template <bool F32>
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
    const float t = -g * (p + q * g2);
    const float s = F32 ? 1.f / (1.f + expf(t)) : __builtin_amdgcn_rcpf(1.f + __expf(t));
    a = g * s;
    da = s + a * (1.f - s) * (p + 3.f * q * g2);
    if (relu) {
      a = g > 0.f ? g : g != g ? g : 0.f;
      da = g > 0.f ? 1.f : 0.f;
    }
  }
};

// An fp32 value as the sum of three bf16 values, each the nearest one to what the
// ones before it leave: 24 bits in all, so the sum is exact, at every exponent
// (below 2^-100 the last terms may lie under the type's smallest normal number).
// The largest values, which would round up to infinity, are cut off instead.
// Infinities and NaN go to the first term alone.
__device__ __forceinline__ void split3(const float (&v)[8], uint4v (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[2] = {v[2 * i], v[2 * i + 1]};
    bool finite[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) finite[k] = fabsf(x[k]) < __builtin_inff();
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t w = pack_bf16(x[0], x[1]);
      if (p == 0) {
        if (finite[0] && (w & 0x7fffu) == 0x7f80u) w = (w & 0xffff0000u) | __float_as_uint(x[0]) >> 16;
        if (finite[1] && (w & 0x7fff0000u) == 0x7f800000u) w = (w & 0xffffu) | (__float_as_uint(x[1]) & 0xffff0000u);
      }
      t[p][i] = w;
      x[0] = finite[0] ? x[0] - __uint_as_float(w << 16) : 0.f;
      x[1] = finite[1] ? x[1] - __uint_as_float(w & 0xffff0000u) : 0.f;
    }
  }
}
// Eight elements to a product's operand: fp32 to three planes.
__device__ __forceinline__ void store_planes(void* p, int64_t off, int64_t plane, const float (&v)[8]) {
  uint4v t[3];
  split3(v, t);
#pragma unroll
  for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4v*>(static_cast<uint16_t*>(p) + off + k * plane) = t[k];
}

// The epilogue on columns [col, col + 8) of one row: v (and for kGate also w,
// the same columns of u; for kActBwd g and u as they lie in memory). oc, og: the
// place in the results and in g and u. Columns from N to pad_to get zeros. fp32
// results that a later product reads are written as its planes (e.plane).
// bf16 g and u are rounded where they are kept (the activation takes them before
// that): the kept state and this epilogue's traffic, which is as long as its
// product at ordinary widths, would double without.
template <bool F32, int EPI>
__device__ __forceinline__ void finish8(const EpiArgs& e, const Activation<F32>& act, int problem, int64_t oc, int64_t og, int col, int N,
                                         float (&v)[8], float (&w)[8], const Raw8<F32>& gr, const Raw8<F32>& ur) {
  const int width = e.pad_to > N ? e.pad_to : N;
  // all but a kStore's rows are padded to whole groups of eight
  const int n = EPI == kStore ? min(8, width - col) : col < width ? 8 : 0;
  if (n <= 0) return;
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
    }
    if (F32 && e.plane)
      store_planes(e.c[0], oc, e.plane, v);
    else
      store8(e.c[0], oc, 8, F32, v);
    if (!F32 && e.c[1]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = bf16_to_f32(f32_to_bf16(v[i]));
        v[i] = fabsf(h) < __builtin_inff() ? v[i] - h : 0.f;
      }
      store8(e.c[1], oc, 8, F32, v);
    }
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
    }
    if (F32) {
      store_planes(e.c[0], oc, e.plane, g);
      store_planes(e.c[1], oc, e.plane, u);
    } else {
      store8(e.c[0], oc, 8, F32, g);
      store8(e.c[1], oc, 8, F32, u);
    }
  }
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
