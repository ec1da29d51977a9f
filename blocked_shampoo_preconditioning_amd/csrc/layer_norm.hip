// Norms before and after a block, fused with gate, dropout and residual
// scale, forward and backward; dropout alone. All are bound by HBM: each pass
// reads every input once and writes every output once, eight elements a lane.
#include "layer_device.h"
#include "layer_kernels.h"

namespace shl {

namespace {

// ------------------------------------------------------------------- dropout
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011). Its 128 bits serve eight elements
// with 16 bits each: the drop probability is a multiple of 2^-16 (the scale
// uses the rounded one, so expectations stay exact), and the integer
// multiplications, a quarter of the rate of other instructions, stay below
// the time of the loads and stores.
__device__ __forceinline__ void drop_factors(const DropArgs& d, uint64_t row, uint32_t c8, float (&m)[8]) {
  uint32_t c0 = c8, c1 = static_cast<uint32_t>(row), c2 = static_cast<uint32_t>(row >> 32), c3 = d.offset;
  uint32_t k0 = d.key0, k1 = d.key1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[2 * i] = (w[i] & 0xffffu) >= d.threshold ? d.scale : 0.f;
    m[2 * i + 1] = (w[i] >> 16) >= d.threshold ? d.scale : 0.f;
  }
}

// A dropped element is 0 whatever its value (also where it is not finite).
__device__ __forceinline__ float dropped(float x, float m) { return m != 0.f ? x * m : 0.f; }

// y = drop(x). Blocks of bx lanes along a row and 256 / bx rows; kRows rows of a
// thread are loaded before any is stored. Bound by HBM: 8192 x 8192 bf16 (268 MB)
// 53 us, 5.0 TB/s, where a large copy reaches 5.3; small ones (257 x 1001 fp32, 2
// MB) by the launch, 4.8 us.
constexpr int kRows = 4;
template <bool F32>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, int bx_log2) {
  const int bx = 1 << bx_log2, by = 256 >> bx_log2;
  const int64_t c8 = static_cast<int64_t>(blockIdx.x) * bx + (threadIdx.x & (bx - 1));
  const int64_t col = c8 * 8;
  if (col >= a.cols) return;
  const int n = static_cast<int>(a.cols - col < 8 ? a.cols - col : 8);
  const int64_t step = static_cast<int64_t>(gridDim.y) * by;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * by + (threadIdx.x >> bx_log2); row < a.rows; row += kRows * step) {
    Raw8<F32> w[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (row + k * step < a.rows) w[k] = fetch8<F32>(a.x, (row + k * step) * a.ldx, static_cast<int>(col), n);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (row + k * step >= a.rows) continue;
      float m[8], v[8];
      drop_factors(a.drop, static_cast<uint64_t>(row + k * step), static_cast<uint32_t>(c8), m);
      unpack8<F32>(settle8<F32>(w[k], static_cast<int>(col), n), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = dropped(v[i], m[i]);
      store8(a.y, (row + k * step) * a.ldy + col, n, F32, v);
    }
  }
}

// --------------------------------------------------------------------- norms
// A workgroup of NT lanes holds a row of up to NT * C * 8 elements in
// registers, so every sum of the row is taken from them and no input is read
// twice. Rows go to workgroups in contiguous ranges: a gate's row stays with
// its workgroup and the backward pass keeps its column sums in registers over
// the range.

// A wave's sum, in a fixed order, through the lanes' own data paths: quads, the
// halves and the whole of a row of 16, then rows 0 to 1 and 2 to 3, 1 to 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += from_lane<0xb1, 0xf>(x);
  x += from_lane<0x4e, 0xf>(x);
  x += from_lane<0x141, 0xf>(x);
  x += from_lane<0x140, 0xf>(x);
  x += from_lane<0x142, 0xa>(x);
  x += from_lane<0x143, 0xc>(x);
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}

// Sum of x and y over the workgroup, in a fixed order. `turn` alternates two
// places, so one barrier a sum is enough.
template <int NT>
__device__ __forceinline__ void block_sum(float& x, float& y, float (&buf)[2][2][NT / 64 + 1], int& turn) {
  x = wave_sum(x);
  y = wave_sum(y);
  if (NT == 64) return;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    buf[turn][0][wave] = x;
    buf[turn][1][wave] = y;
  }
  // only LDS is shared here: loads and stores to memory stay in flight
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  x = y = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    x += buf[turn][0][w];
    y += buf[turn][1][w];
  }
  turn ^= 1;
}

// Row-uniform statistics of v (C chunks of eight a lane): mean (0 for RMS) and
// 1 / sqrt(mean square + eps). Lanes past the row hold zeros; the centred
// squares of a layer norm are summed in a second sweep over the registers,
// which loses no digits to a large mean.
template <int NT, int C>
__device__ __forceinline__ void row_stats(const float (&v)[C][8], const int (&n)[C], int kind, int d, float eps, float& mean,
                                          float& rstd, float (&buf)[2][2][NT / 64 + 1], int& turn) {
  mean = 0.f;
  float s = 0.f, q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[c][i], q += v[c][i] * v[c][i];
  block_sum<NT>(s, q, buf, turn);
  if (kind == kNormLayer) {
    mean = s / d;
    q = 0.f;
    float unused = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = i < n[c] ? v[c][i] - mean : 0.f;
        q += t * t;
      }
    block_sum<NT>(q, unused, buf, turn);
  }
  rstd = 1.f / sqrtf(q / d + eps);
}

// A lane's chunks of a row, as fetch8 leaves them, and their values.
template <bool F32, int C, int NT, bool GENERAL>
__device__ __forceinline__ void fetch(const void* p, int64_t off, const int (&n)[C], Raw8<F32> (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * NT + threadIdx.x) * 8;
    if (GENERAL)
      v[c] = fetch8<F32>(p, off, col, n[c]);
    else if (n[c] > 0)
      v[c] = fetch8<F32>(p, off, col, 8);
    else
      v[c] = Raw8<F32>{};
  }
}
template <bool F32, int C, int NT, bool GENERAL>
__device__ __forceinline__ void unpack(const Raw8<F32> (&w)[C], const int (&n)[C], float (&v)[C][8]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
    unpack8<F32>(GENERAL ? settle8<F32>(w[c], (c * NT + static_cast<int>(threadIdx.x)) * 8, n[c]) : w[c], v[c]);
}
// The same of a vector that may not be there (`none` stands for its elements).
template <bool F32, int C, int NT, bool GENERAL>
__device__ __forceinline__ void fetch_vec(const void* p, int64_t off, const int (&n)[C], Raw8<F32> (&v)[C]) {
  if (p) fetch<F32, C, NT, GENERAL>(p, off, n, v);
}
template <bool F32, int C, int NT, bool GENERAL>
__device__ __forceinline__ void unpack_vec(const void* p, const Raw8<F32> (&w)[C], const int (&n)[C], float none, float (&v)[C][8]) {
  if (p) {
    unpack<F32, C, NT, GENERAL>(w, n, v);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = none;
  }
}
template <bool F32, int C, int NT, bool GENERAL>
__device__ __forceinline__ void load_vec(const void* p, int64_t off, const int (&n)[C], float none, float (&v)[C][8]) {
  Raw8<F32> w[C];
  fetch_vec<F32, C, NT, GENERAL>(p, off, n, w);
  unpack_vec<F32, C, NT, GENERAL>(p, w, n, none, v);
}
template <int C>
__device__ __forceinline__ void fill(float (&v)[C][8], float x) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = x;
}
template <int C, int NT, bool GENERAL>
__device__ __forceinline__ void store_row(void* p, int64_t off, const int (&n)[C], bool f32, const float (&v)[C][8]) {
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (n[c] > 0) store8(p, off + (c * NT + threadIdx.x) * 8, GENERAL ? n[c] : 8, f32, v[c]);
}

// Lanes past a row's end hold zeros: n is what a chunk has of the row (0..8).
template <int C, int NT>
__device__ __forceinline__ void chunk_sizes(int d, int (&n)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) n[c] = max(0, min(8, d - static_cast<int>(c * NT + threadIdx.x) * 8));
}

// p = norm(z) w + b, r = alpha x + drop(gate p), n = norm'(r) w' + b': reads x and
// z, writes r, n and four statistics a row. GENERAL: there is a bias, or the
// row's last group is short; without, the registers for them are saved. 16384 x
// 2048 bf16, RMS, gate, dropout (268 MB): 54 us, 5.0 TB/s, bound by HBM; 3001 x
// 777 fp32, layer norms (37 MB): 17.5 us, bound by the launch, the first loads (4
// us for all rows at once) and two rows of a workgroup one after the other (one
// row each 18 us, three 20, rows of one wave 18); one row of 2048: 3.6 us, the
// launch.
template <bool F32, int NT, int C, bool GENERAL>
__global__ __launch_bounds__(NT) void norm_forward_kernel(NormArgs a) {
  __shared__ float buf[2][2][NT / 64 + 1];
  int turn = 0;
  const int64_t per = (a.rows + gridDim.x - 1) / gridDim.x;
  const int64_t first = blockIdx.x * per, last = first + per < a.rows ? first + per : a.rows;
  if (first >= last) return;
  int n[C];
  chunk_sizes<C, NT>(a.d, n);
  Raw8<F32> xr[C], zr[C];
  fetch<F32, C, NT, GENERAL>(a.x, first * a.ldx, n, xr);
  if (a.z) fetch<F32, C, NT, GENERAL>(a.z, first * a.ldz, n, zr);
  float wp[C][8], bp[C][8], gate[C][8], wn[C][8], bn[C][8];
  // the first gate row is loaded with the weights, not when a row waits for it
  int64_t group = first / a.rows_per_gate;
  {
    Raw8<F32> v[5][C];
    fetch_vec<F32, C, NT, GENERAL>(a.w_post, 0, n, v[0]);
    fetch_vec<F32, C, NT, GENERAL>(a.w_next, 0, n, v[1]);
    if (GENERAL) {
      fetch_vec<F32, C, NT, GENERAL>(a.b_post, 0, n, v[2]);
      fetch_vec<F32, C, NT, GENERAL>(a.b_next, 0, n, v[3]);
    }
    fetch_vec<F32, C, NT, GENERAL>(a.gate, group * a.ld_gate, n, v[4]);
    unpack_vec<F32, C, NT, GENERAL>(a.w_post, v[0], n, 1.f, wp);
    unpack_vec<F32, C, NT, GENERAL>(a.w_next, v[1], n, 1.f, wn);
    if (GENERAL) {
      unpack_vec<F32, C, NT, GENERAL>(a.b_post, v[2], n, 0.f, bp);
      unpack_vec<F32, C, NT, GENERAL>(a.b_next, v[3], n, 0.f, bn);
    }
    unpack_vec<F32, C, NT, GENERAL>(a.gate, v[4], n, 1.f, gate);
  }
  for (int64_t row = first; row < last; ++row) {
    float z[C][8], r[C][8];
    unpack<F32, C, NT, GENERAL>(xr, n, r);
    unpack<F32, C, NT, GENERAL>(zr, n, z);
    if (row + 1 < last) {  // the next row's loads go ahead of this row's stores
      fetch<F32, C, NT, GENERAL>(a.x, (row + 1) * a.ldx, n, xr);
      if (a.z) fetch<F32, C, NT, GENERAL>(a.z, (row + 1) * a.ldz, n, zr);
    }
    float mz = 0.f, rz = 1.f, mr = 0.f, rr = 1.f;
    if (a.z) {
      if (a.gate && row >= (group + 1) * a.rows_per_gate) {
        group = row / a.rows_per_gate;
        load_vec<F32, C, NT, GENERAL>(a.gate, group * a.ld_gate, n, 1.f, gate);
      }
      if (a.post_kind != kNormNone) row_stats<NT, C>(z, n, a.post_kind, a.d, a.eps, mz, rz, buf, turn);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = 1.f;
        if (a.drop.threshold) drop_factors(a.drop, row, c * NT + threadIdx.x, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float p = (z[c][i] - mz) * rz * wp[c][i];
          if (GENERAL) p += bp[c][i];
          r[c][i] = i < n[c] ? a.alpha * r[c][i] + dropped(gate[c][i] * p, m[i]) : 0.f;
        }
      }
      store_row<C, NT, GENERAL>(a.r, row * a.ldr, n, F32, r);
    }
    if (a.next_kind != kNormNone) {
      row_stats<NT, C>(r, n, a.next_kind, a.d, a.eps, mr, rr, buf, turn);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[c][i] = (r[c][i] - mr) * rr * wn[c][i];
          if (GENERAL) r[c][i] += bn[c][i];
        }
      store_row<C, NT, GENERAL>(a.n, row * a.ldn, n, F32, r);
    }
    if (a.stats && threadIdx.x == 0) {
      const floatx4 s = {mz, rz, mr, rr};
      *reinterpret_cast<floatx4*>(a.stats + row * 4) = s;
    }
  }
}

// The second term of bf16 n: what its rounding left. An element counts only where
// the rounding of what is made again here is n's element itself, so that n may
// have been changed since, and every other input too: the term is then 0. Bound by
// HBM: 4096 x 768 (19 MB) in 6 us.
__global__ __launch_bounds__(256) void norm_rest_kernel(NormArgs a, uint16_t* out, int64_t ld_out) {
  const int64_t c8 = ld_out / 8, total = c8 * a.rows;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / c8;
    const int col = static_cast<int>(i - row * c8) * 8, m = max(0, min(8, a.d - col));
    const floatx4 st = *reinterpret_cast<const floatx4*>(a.stats + row * 4);
    Raw8<false> xr = fetch8<false>(a.x, row * a.ldx, col, m), nr = fetch8<false>(a.n, row * a.ldn, col, m), wr, br;
    if (a.w_next) wr = fetch8<false>(a.w_next, 0, col, m);
    if (a.b_next) br = fetch8<false>(a.b_next, 0, col, m);
    float x[8], n[8], w[8], b[8];
    unpack8<false>(settle8<false>(xr, col, m), x);
    unpack8<false>(settle8<false>(nr, col, m), n);
    if (a.w_next) unpack8<false>(settle8<false>(wr, col, m), w);
    if (a.b_next) unpack8<false>(settle8<false>(br, col, m), b);
    uint4v t;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float d[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 2 * k + h;
        float v = (x[e] - st[2]) * st[3];
        if (a.w_next) v *= w[e];
        if (a.b_next) v += b[e];
        const float rounded = bf16_to_f32(f32_to_bf16(v));
        d[h] = e < m && rounded == n[e] && fabsf(v) < __builtin_inff() ? v - rounded : 0.f;
      }
      t[k] = pack_bf16(d[0], d[1]);
    }
    *reinterpret_cast<uint4v*>(out + row * ld_out + col) = t;
  }
}

// Backward. With c = dn w', dR = dr + rstd (c - [mean c] - r^ mean(c r^));
// dx = alpha dR; db = drop(dR); dgate = sum db p; dp = db gate; dz likewise
// from dp w. The four vectors' sums stay in registers over the workgroup's
// rows and go to partial[vector][workgroup][d]; norm_sums_kernel joins them in
// order. A gate row whose tokens all lie in this range is stored at once; one
// that reaches over an end of the range goes to the partial sums (place 0: it
// began before the range or fills it, place 1: it goes on after it). r^ is taken
// from r as it was rounded, since r is what is kept (the gradients of next's
// vectors are off by 0.0023 in norm, by their own rounding 0.0017). 16384 x
// 2048 bf16 (403 MB): 83 us, 4.9 TB/s, bound by HBM; 3001 x 777 fp32 (56 MB): 23
// us, as the forward pass.
enum { kSumWNext = 0, kSumBNext = 1, kSumWPost = 2, kSumBPost = 3, kSumGate = 4, kSums = 6 };

template <bool F32, int NT, int C, bool GENERAL>
__global__ __launch_bounds__(NT, NT == 512 || GENERAL ? 2 : 3) void norm_backward_kernel(NormArgs a) {
  __shared__ float buf[2][2][NT / 64 + 1];
  int turn = 0;
  const int64_t per = (a.rows + gridDim.x - 1) / gridDim.x;
  const int64_t first = blockIdx.x * per, last = first + per < a.rows ? first + per : a.rows;
  int n[C];
  chunk_sizes<C, NT>(a.d, n);
  const bool has_next = a.next_kind != kNormNone;
  Raw8<F32> rw[C], dnw[C], drw[C], zw[C];
  floatx4 st;
  auto load = [&](int64_t row) {
    st = *reinterpret_cast<const floatx4*>(a.stats + row * 4);
    if (has_next) {
      fetch<F32, C, NT, GENERAL>(a.r, row * a.ldr, n, rw);
      fetch<F32, C, NT, GENERAL>(a.dn, row * a.lddn, n, dnw);
    }
    if (a.dr) fetch<F32, C, NT, GENERAL>(a.dr, row * a.lddr, n, drw);
    if (a.z) fetch<F32, C, NT, GENERAL>(a.z, row * a.ldz, n, zw);
  };
  if (first < last) load(first);
  // Rows over 4096 wide read weights and gate anew for each row (from the
  // caches): even so fp32 spills 35 registers of a lane, with GENERAL 129 (bf16
  // 89), and 1024 lanes a row would have half as many each (not tried: 8192 x 8192
  // both norms RMS bf16 222 us, 3.6 TB/s, layer norms with biases 653).
  constexpr bool HOLD = C == 1;
  float wp[C][8], bp[C][8], gate[C][8], wn[C][8];
  auto load_next = [&]() { load_vec<F32, C, NT, GENERAL>(a.w_next, 0, n, 1.f, wn); };
  auto load_post = [&]() {
    load_vec<F32, C, NT, GENERAL>(a.w_post, 0, n, 1.f, wp);
    if (GENERAL) load_vec<F32, C, NT, GENERAL>(a.b_post, 0, n, 0.f, bp);
  };
  int64_t group = first / a.rows_per_gate;
  fill<C>(gate, 1.f);
  if (HOLD && first < last) {  // the first gate row too
    Raw8<F32> v[4][C];
    fetch_vec<F32, C, NT, GENERAL>(a.w_next, 0, n, v[0]);
    fetch_vec<F32, C, NT, GENERAL>(a.w_post, 0, n, v[1]);
    if (GENERAL) fetch_vec<F32, C, NT, GENERAL>(a.b_post, 0, n, v[2]);
    fetch_vec<F32, C, NT, GENERAL>(a.gate, group * a.ld_gate, n, v[3]);
    unpack_vec<F32, C, NT, GENERAL>(a.w_next, v[0], n, 1.f, wn);
    unpack_vec<F32, C, NT, GENERAL>(a.w_post, v[1], n, 1.f, wp);
    if (GENERAL) unpack_vec<F32, C, NT, GENERAL>(a.b_post, v[2], n, 0.f, bp);
    unpack_vec<F32, C, NT, GENERAL>(a.gate, v[3], n, 1.f, gate);
  }
  float s_wn[C][8], s_bn[C][8], s_wp[C][8], s_bp[C][8], s_g[C][8];
  fill<C>(s_wn, 0.f);
  fill<C>(s_wp, 0.f);
  fill<C>(s_g, 0.f);
  if (GENERAL) {
    fill<C>(s_bn, 0.f);
    fill<C>(s_bp, 0.f);
  }
  const int64_t plane = static_cast<int64_t>(gridDim.x) * a.d;
  auto put = [&](int what, const float (&v)[C][8]) {
    store_row<C, NT, GENERAL>(a.partial + what * plane, static_cast<int64_t>(blockIdx.x) * a.d, n, true, v);
  };
  auto put_gate = [&]() {
    const int64_t begin = group * a.rows_per_gate;
    const int64_t end = begin + a.rows_per_gate < a.rows ? begin + a.rows_per_gate : a.rows;
    if (begin >= first && end <= last) {
      store_row<C, NT, GENERAL>(a.dgate, group * a.ld_dgate, n, F32, s_g);
    } else {
      put(kSumGate + (begin <= first ? 0 : 1), s_g);
    }
  };
  const float inv_d = 1.f / a.d;
  for (int64_t row = first; row < last; ++row) {
    float r[C][8], dn[C][8], dr[C][8], z[C][8];
    const float m = st[2], rs = st[3], mz = st[0], rz = st[1];
    if (has_next) {
      unpack<F32, C, NT, GENERAL>(rw, n, r);
      unpack<F32, C, NT, GENERAL>(dnw, n, dn);
    }
    if (a.dr)
      unpack<F32, C, NT, GENERAL>(drw, n, dr);
    else
      fill<C>(dr, 0.f);
    if (a.z) unpack<F32, C, NT, GENERAL>(zw, n, z);
    if (row + 1 < last) load(row + 1);  // ahead of this row's stores
    if (a.gate && row >= (group + 1) * a.rows_per_gate) {
      if (a.dgate) {
        put_gate();
        fill<C>(s_g, 0.f);
      }
      group = row / a.rows_per_gate;
      if (HOLD) load_vec<F32, C, NT, GENERAL>(a.gate, group * a.ld_gate, n, 1.f, gate);
    }
    if (has_next) {
      if (!HOLD) load_next();
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[c][i] = i < n[c] ? (r[c][i] - m) * rs : 0.f;  // r^
          s_wn[c][i] += dn[c][i] * r[c][i];
          if (GENERAL) s_bn[c][i] += dn[c][i];
          dn[c][i] *= wn[c][i];
          s1 += dn[c][i];
          s2 += dn[c][i] * r[c][i];
        }
      block_sum<NT>(s1, s2, buf, turn);
      s1 = a.next_kind == kNormLayer ? s1 * inv_d : 0.f;
      s2 *= inv_d;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dr[c][i] += rs * (dn[c][i] - s1 - r[c][i] * s2);
    }
    if (a.dx) {
      float o[C][8];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[c][i] = a.alpha * dr[c][i];
      store_row<C, NT, GENERAL>(a.dx, row * a.lddx, n, F32, o);
    }
    if (a.z) {
      if (!HOLD) {
        load_post();
        if (a.gate) load_vec<F32, C, NT, GENERAL>(a.gate, group * a.ld_gate, n, 1.f, gate);
      }
      float t1 = 0.f, t2 = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float mk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mk[i] = 1.f;
        if (a.drop.threshold) drop_factors(a.drop, row, c * NT + threadIdx.x, mk);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float zh = i < n[c] ? (z[c][i] - mz) * rz : 0.f;
          const float db = i < n[c] ? dropped(dr[c][i], mk[i]) : 0.f;
          float p = zh * wp[c][i];
          if (GENERAL) p += bp[c][i];
          s_g[c][i] += db * p;
          const float dp = db * gate[c][i];
          s_wp[c][i] += dp * zh;
          if (GENERAL) s_bp[c][i] += dp;
          z[c][i] = zh;
          dr[c][i] = dp * wp[c][i];
          t1 += dr[c][i];
          t2 += dr[c][i] * zh;
        }
      }
      if (a.post_kind != kNormNone) {
        block_sum<NT>(t1, t2, buf, turn);
        t1 = a.post_kind == kNormLayer ? t1 * inv_d : 0.f;
        t2 *= inv_d;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) dr[c][i] = rz * (dr[c][i] - t1 - z[c][i] * t2);
      }
      if (a.dz) store_row<C, NT, GENERAL>(a.dz, row * a.lddz, n, F32, dr);
    }
  }
  if (a.dw_next) put(kSumWNext, s_wn);
  if (a.dw_post) put(kSumWPost, s_wp);
  if (GENERAL) {
    if (a.db_next) put(kSumBNext, s_bn);
    if (a.db_post) put(kSumBPost, s_bp);
  }
  if (a.gate && a.dgate && first < last) put_gate();
}

// Joins the workgroups' column sums: 32 columns a workgroup, its 32 half-waves
// take the parts in turn with eight loads in flight, and the 32 sums are added
// in order. Bound by the launch and two trips to memory: three vectors of 2048
// from 745 parts 5.9 us (7.0 with 64-bit indexes; four loads 7.2, sixteen 6.0).
// blockIdx.y: the vectors of `what`; then the gate's rows that reach over an end
// of a range: each row in turn (by_row), or for more rows than ends each end,
// where the first one that a row reaches over stands for it.
struct SumList {
  int32_t n;
  int32_t what[4];
  int32_t by_row;
};
__global__ __launch_bounds__(1024) void norm_sums_kernel(NormArgs a, int parts, SumList list) {
  __shared__ float sums[32][33];
  const int c32 = threadIdx.x & 31, slot = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c32;
  const int64_t per = parts ? (a.rows + parts - 1) / parts : 1;
  const int64_t plane = static_cast<int64_t>(parts) * a.d;
  void* out;
  int64_t at = 0;
  int64_t lo = 0, hi = parts, begin = -1;
  const float* p;
  if (static_cast<int>(blockIdx.y) < list.n) {
    const int what = list.what[blockIdx.y];
    out = what == kSumWNext ? a.dw_next : what == kSumBNext ? a.db_next : what == kSumWPost ? a.dw_post : a.db_post;
    p = a.partial + what * plane;
  } else {
    const int64_t k = blockIdx.y - list.n;
    int64_t group = k;
    if (!list.by_row) {
      if ((k + 1) * per >= a.rows) return;
      group = (k + 1) * per / a.rows_per_gate;
    }
    begin = group * a.rows_per_gate;
    const int64_t end = begin + a.rows_per_gate < a.rows ? begin + a.rows_per_gate : a.rows;
    lo = begin / per;
    hi = (end + per - 1) / per;
    if (hi - lo <= 1 || (!list.by_row && lo != k)) return;
    out = a.dgate;
    at = group * a.ld_dgate;
    p = a.partial + kSumGate * plane;
  }
  // A gate row's first part is in place 1 if the row began in its range. Indexes
  // stay under 2^32: a part's lanes hold eight columns each, and all parts' lanes
  // are resident at once.
  const uint32_t other = begin > lo * per ? static_cast<uint32_t>(plane) : 0u, step = 32u * a.d;
  float s = 0.f;
  if (col < a.d) {
    uint32_t at_k = static_cast<uint32_t>(lo + slot) * a.d + col;
    for (int k = static_cast<int>(lo) + slot; k < hi; k += 256, at_k += 8 * step) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = k + 32 * i < hi ? p[at_k + i * step + (k + 32 * i == lo ? other : 0u)] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i];
    }
  }
  sums[slot][c32] = s;
  __syncthreads();
  if (slot == 0 && col < a.d) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += sums[w][c32];
    if (a.f32)
      static_cast<float*>(out)[at + col] = s;
    else
      static_cast<uint16_t*>(out)[at + col] = f32_to_bf16(s);
  }
}

int norm_lanes(int d) { return d <= 512 ? 64 : d <= 1024 ? 128 : d <= 2048 ? 256 : 512; }

bool norm_general(const NormArgs& a, bool backward) {
  return a.d % 8 != 0 || a.b_post || (backward ? a.db_post || a.db_next : a.b_next != nullptr);
}

// Workgroups of the row kernels: as many as the card holds at once (four times
// that in the forward pass: 16384 x 2048 54 us, 56 at twice and at once; backward
// at three waves a SIMD 95, 116 at two and at four), and where there are rows
// enough at least two rows each (forward) or four, which share the reads of
// weights and keep the backward pass's column sums a small part of its traffic
// (3001 x 777 fp32 backward with its sums: 29 us at four rows, 28 at three, 34 at
// six; 4096 x 768 bf16 22 at four, 24 at three and at six).
int64_t norm_grid(const NormArgs& a, bool backward, bool general) {
  const int lanes = norm_lanes(a.d);
  const int64_t most = backward ? 256 * (lanes == 512 || general ? 8 : 12) * 64 / lanes : 4 * 256 * 16 * 64 / lanes;
  int64_t per = (a.rows + most - 1) / most;
  const int64_t wanted = backward ? 4 : 2;
  const int64_t least = (a.rows + 511) / 512;
  const int64_t few = least < wanted ? least : wanted;
  if (per < few) per = few;
  return per ? (a.rows + per - 1) / per : 0;
}

template <bool F32, int NT, int C>
void launch_norm(const NormArgs& a, bool backward, int64_t grid, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(grid)), b(NT);
  const bool general = norm_general(a, backward);
  if (backward && general)
    hipLaunchKernelGGL((norm_backward_kernel<F32, NT, C, true>), g, b, 0, s, a);
  else if (backward)
    hipLaunchKernelGGL((norm_backward_kernel<F32, NT, C, false>), g, b, 0, s, a);
  else if (general)
    hipLaunchKernelGGL((norm_forward_kernel<F32, NT, C, true>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((norm_forward_kernel<F32, NT, C, false>), g, b, 0, s, a);
}

template <bool F32>
hipError_t dispatch_norm(const NormArgs& a, bool backward, int64_t grid, hipStream_t s) {
  if (a.d > kMaxNormWidth) return hipErrorInvalidValue;
  switch (norm_lanes(a.d)) {
    case 64: launch_norm<F32, 64, 1>(a, backward, grid, s); break;
    case 128: launch_norm<F32, 128, 1>(a, backward, grid, s); break;
    case 256: launch_norm<F32, 256, 1>(a, backward, grid, s); break;
    default:
      if (a.d <= 4096)
        launch_norm<F32, 512, 1>(a, backward, grid, s);
      else
        launch_norm<F32, 512, 2>(a, backward, grid, s);
  }
  return hipGetLastError();
}

}  // namespace

// An upper bound that goes by the sizes alone.
int64_t norm_partial_floats(const NormArgs& a) { return kSums * norm_grid(a, true, false) * a.d; }

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return a.f32 ? dispatch_norm<true>(a, false, norm_grid(a, false, norm_general(a, false)), s)
               : dispatch_norm<false>(a, false, norm_grid(a, false, norm_general(a, false)), s);
}

hipError_t launch_norm_rest(const NormArgs& a, uint16_t* out, int64_t ld_out, hipStream_t s) {
  const int64_t blocks = (a.rows * (ld_out / 8) + 255) / 256;
  if (blocks == 0) return hipSuccess;
  if (a.f32) return hipErrorInvalidValue;
  hipLaunchKernelGGL(norm_rest_kernel, dim3(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a, out, ld_out);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
  const int64_t grid = norm_grid(a, true, norm_general(a, true));
  if (grid) {
    const hipError_t e = a.f32 ? dispatch_norm<true>(a, true, grid, s) : dispatch_norm<false>(a, true, grid, s);
    if (e != hipSuccess) return e;
  }
  SumList list{};
  if (a.dw_next) list.what[list.n++] = kSumWNext;
  if (a.db_next) list.what[list.n++] = kSumBNext;
  if (a.dw_post) list.what[list.n++] = kSumWPost;
  if (a.db_post) list.what[list.n++] = kSumBPost;
  int64_t ends = 0;
  if (a.dgate && grid > 1) {
    const int64_t groups = (a.rows + a.rows_per_gate - 1) / a.rows_per_gate;
    list.by_row = groups <= grid - 1;
    ends = list.by_row ? groups : grid - 1;
  }
  if (list.n + ends == 0) return hipSuccess;
  hipLaunchKernelGGL(norm_sums_kernel, dim3((a.d + 31) / 32, static_cast<uint32_t>(list.n + ends)), dim3(1024), 0, s, a,
                     static_cast<int>(grid), list);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  const int64_t c8 = (a.cols + 7) / 8;
  int log2 = 0;
  while (log2 < 8 && (1 << log2) < c8) ++log2;
  const int64_t gx = (c8 + (1 << log2) - 1) >> log2, by = 256 >> log2;
  int64_t gy = (a.rows + by - 1) / by;
  const int64_t want = (gy + kRows - 1) / kRows;
  gy = want < 32768 ? want : 32768;
  if (gx > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(gx), static_cast<uint32_t>(gy));
  if (a.f32)
    hipLaunchKernelGGL(dropout_kernel<true>, grid, dim3(256), 0, s, a, log2);
  else
    hipLaunchKernelGGL(dropout_kernel<false>, grid, dim3(256), 0, s, a, log2);
  return hipGetLastError();
}

}  // namespace shl
