// Operands of the 8-bit products.
//
// A block of 128 values has the scale 2^e, e the smallest exponent (-126 at
// least) with max |x| <= 448 * 2^e, and holds x / 2^e as e4m3, to nearest even.
// Division by a power of two is exact, so the one rounding is the value's own and
// no order of operations shows in the result. An infinite or NaN element becomes
// NaN and takes no part in the maximum.
//
// A workgroup has a tile of 128 x 128: 256 threads with eight rows and eight
// columns each, loaded at once and kept in registers, so that one read of x gives
// the values by rows, by columns or both. What comes by columns is transposed
// through LDS. Memory bounds it: 2 or 4 bytes in, 1 or 2 out an element. For that the
// maxima are taken of two bf16 magnitudes a word, and the conversion divides.
#include "experts_device.h"

namespace she {

using shl::fetch8;
using shl::Raw8;
using shl::settle8;

namespace {

constexpr int kThreads = 256;

// Magnitudes of a thread's elements, for maxima: fp32 one a word, bf16 two.
typedef __attribute__((ext_vector_type(2))) unsigned short ushort2v;
template <bool F32>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
  if (F32) return max(a, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, a), __builtin_bit_cast(ushort2v, b)));
}
template <bool F32>
__device__ __forceinline__ uint32_t word_magnitude(uint32_t w) { return w & (F32 ? 0x7fffffffu : 0x7fff7fffu); }
// The same with 0 for what is not finite.
template <bool F32>
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w) {
  if (F32) return magnitude(__uint_as_float(w));
  return magnitude(__uint_as_float(w & 0xffff0000u)) | magnitude(__uint_as_float(w << 16)) >> 16;
}
// A word's elements as magnitude bits of fp32.
template <bool F32>
__device__ __forceinline__ uint32_t first_of(uint32_t w) { return F32 ? w : w << 16; }
__device__ __forceinline__ uint32_t second_of(uint32_t w) { return w & 0xffff0000u; }

template <int CTRL, bool F32>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return word_max<F32>(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
// The largest of 16 lanes, in all of them (rotations of a row of 16).
template <bool F32>
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = dpp_max<0x128, F32>(v);
  v = dpp_max<0x124, F32>(v);
  v = dpp_max<0x122, F32>(v);
  return dpp_max<0x121, F32>(v);
}

// The expert whose rows block p holds (-1 where p is behind all blocks), its first
// block, row tile and row, its rows, and the totals. Every wave finds it by itself.
struct Found {
  int expert, block0, tile0, row0, rows;
  int all_tiles, all_rows;
};
__device__ __forceinline__ Found find_group(const Groups& g, int p, int tile_blocks, int32_t* first_block) {
  const int lane = threadIdx.x & 63, each = (g.experts + 63) / 64;
  const int from = min(lane * each, g.experts), to = min(from + each, g.experts);
  auto blocks_of = [&](int lo, int hi) { return hi > lo ? (hi - lo + kBlock - 1) / kBlock : 0; };
  const int begin = group_row(g, from);
  int blocks = 0, tiles = 0, lo = begin;
  for (int e = from; e < to; ++e) {
    const int hi = group_row(g, e + 1), b = blocks_of(lo, hi);
    blocks += b;
    tiles += (b + tile_blocks - 1) / tile_blocks;
    lo = hi;
  }
  Found f{-1, 0, 0, 0, 0, 0, __shfl(lo, 63)};
  int pb = blocks, pt = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int ub = __shfl_up(pb, d), ut = __shfl_up(pt, d);
    if (lane >= d) pb += ub, pt += ut;
  }
  f.all_tiles = __shfl(pt, 63);
  if (first_block && lane == 63) first_block[g.experts] = min(pb, g.blocks);
  const bool here = p >= pb - blocks && p < pb;
  pb -= blocks, pt -= tiles;
  lo = begin;
  for (int e = from; e < to; ++e) {
    const int hi = group_row(g, e + 1), b = blocks_of(lo, hi);
    if (first_block) first_block[e] = min(pb, g.blocks);
    if (p >= pb && p < pb + b) f.expert = e, f.block0 = pb, f.tile0 = pt, f.row0 = lo, f.rows = hi - lo;
    pb += b;
    pt += (b + tile_blocks - 1) / tile_blocks;
    lo = hi;
  }
  const uint64_t found = __ballot(here);
  const int who = found ? __ffsll(static_cast<unsigned long long>(found)) - 1 : 0;
  f.expert = found ? __builtin_amdgcn_readlane(f.expert, who) : -1;
  f.block0 = __builtin_amdgcn_readlane(f.block0, who);
  f.tile0 = __builtin_amdgcn_readlane(f.tile0, who);
  f.row0 = __builtin_amdgcn_readlane(f.row0, who);
  f.rows = __builtin_amdgcn_readlane(f.rows, who);
  return f;
}

// A thread's part of a tile: eight rows of eight columns.
template <bool F32>
struct Tile {
  static constexpr int W = F32 ? 8 : 4;
  Eight<F32> v[8];

  // Eight rows' bytes of column c over its scale.
  __device__ __forceinline__ uint2 column(int c, float scale) const {
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (F32) {
        o[h] = pack2<false>(0, __uint_as_float(v[4 * h].w[c]), __uint_as_float(v[4 * h + 1].w[c]), scale);
        o[h] = pack2<true>(o[h], __uint_as_float(v[4 * h + 2].w[c]), __uint_as_float(v[4 * h + 3].w[c]), scale);
      } else {
        const uint32_t pick = c & 1 ? 0x07060302u : 0x05040100u;  // the same column of two rows, the lower row's low
        o[h] = pack2_bf16<false>(0, __builtin_amdgcn_perm(v[4 * h + 1].w[c / 2], v[4 * h].w[c / 2], pick), scale);
        o[h] = pack2_bf16<true>(o[h], __builtin_amdgcn_perm(v[4 * h + 3].w[c / 2], v[4 * h + 2].w[c / 2], pick), scale);
      }
    }
    return uint2{o[0], o[1]};
  }
};

// A thread's magnitudes and their largest by column. Words that hold something not
// finite, which is rare, are looked at again.
template <bool F32>
__device__ __forceinline__ void tile_magnitudes(const Tile<F32>& t, uint32_t (&m)[8][Tile<F32>::W], uint32_t (&top)[Tile<F32>::W]) {
  constexpr int W = Tile<F32>::W;
  auto maxima = [&]() {
    uint32_t all = 0;
#pragma unroll
    for (int c = 0; c < W; ++c) {
      top[c] = m[0][c];
#pragma unroll
      for (int i = 1; i < 8; ++i) top[c] = word_max<F32>(top[c], m[i][c]);
      all = word_max<F32>(all, top[c]);
    }
    return all;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < W; ++c) m[i][c] = word_magnitude<F32>(t.v[i].w[c]);
  const uint32_t all = maxima();
  if (__any(first_of<F32>(all) >= 0x7f800000u || (!F32 && all >= 0x7f800000u))) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < W; ++c) m[i][c] = finite_magnitude<F32>(t.v[i].w[c]);
    maxima();
  }
}

// The values by columns go out transposed, through LDS.
template <bool F32>
__device__ __forceinline__ void write_columns(const Tile<F32>& t, const uint32_t (&scale)[8], char* lds, uint8_t* out, int64_t pitch, int rows) {
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint2*>(lds + (cg * 8 + c) * 128 + (((rt >> 1) ^ (cg & 7)) << 4) + (rt & 1) * 8) = t.column(c, value_of(scale[c]));
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int col = (threadIdx.x >> 3) + 32 * k, chunk = threadIdx.x & 7;
    const shl::uint4v v = *reinterpret_cast<const shl::uint4v*>(lds + col * 128 + ((chunk ^ ((col >> 3) & 7)) << 4));
    if (col < rows) __builtin_memcpy(out + col * pitch + chunk * 16, &v, 16);
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a) {
  constexpr int W = Tile<F32>::W;
  __shared__ __attribute__((aligned(16))) char lds[128 * 128];
  __shared__ uint32_t tops[4][128];
  const int p = static_cast<int>(blockIdx.x / a.col_blocks), kt = static_cast<int>(blockIdx.x - static_cast<uint32_t>(p) * a.col_blocks);
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  int row0 = p * kBlock, count = min(kBlock, a.g.n - row0);
  if (a.g.offsets) {
    const bool lead = kt == 0 && p == 0;
    const Found f = find_group(a.g, p, a.tile_blocks, lead && threadIdx.x < 64 ? a.first_block : nullptr);
    if (lead && a.tiles) {
      // tiles behind the experts': rows that get zeros
      const int tile_rows = a.tile_blocks * kBlock, rest = a.g.n - f.all_rows;
      const int more = (rest + tile_rows - 1) / tile_rows;
      for (int i = threadIdx.x; i < more; i += kThreads)
        if (f.all_tiles + i < a.max_tiles)
          a.tiles[f.all_tiles + i] = RowTile{-1, 0, f.all_rows + i * tile_rows, min(tile_rows, rest - i * tile_rows)};
      if (threadIdx.x == 0) *a.tile_count = min(f.all_tiles + more, a.max_tiles);
    }
    if (f.expert < 0) return;
    const int local = p - f.block0;
    row0 = f.row0 + local * kBlock;
    count = min(kBlock, f.rows - local * kBlock);
    if (kt == 0 && threadIdx.x == 0 && a.tiles && local % a.tile_blocks == 0) {
      const int at = f.tile0 + local / a.tile_blocks;
      if (at < a.max_tiles) a.tiles[at] = RowTile{f.expert, p, row0, min(a.tile_blocks * kBlock, f.rows - local * kBlock)};
    }
  }
  const int col = kt * kBlock + cg * 8, n = min(8, max(0, a.cols - col));
  Raw8<F32> raw[8];
  int64_t at[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rt * 8 + i;
    int64_t from = row0 + r;
    if (a.source && r < count) {
      const int32_t s = a.source[row0 + r];
      from = min(static_cast<uint32_t>(s < 0 ? ~s : s) / a.slots, static_cast<uint32_t>(a.rows_in - 1));
    }
    at[i] = from * a.ld;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i] = fetch8<F32>(a.x, at[i], col, rt * 8 + i < count ? n : 0);
  Tile<F32> t;
#pragma unroll
  for (int i = 0; i < 8; ++i) t.v[i] = Eight<F32>(settle8<F32>(raw[i], col, rt * 8 + i < count ? n : 0));
  uint32_t m[8][W], top[W];
  tile_magnitudes<F32>(t, m, top);

  if (a.by_rows) {
    const int64_t pitch = static_cast<int64_t>(a.col_blocks) * kBlock;
    uint8_t* out = a.by_rows + (static_cast<int64_t>(p) * kBlock + rt * 8) * pitch + col;
    uint8_t* scales = a.row_scales + (static_cast<int64_t>(kt) * a.g.blocks + p) * kBlock;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w = m[i][0];
#pragma unroll
      for (int c = 1; c < W; ++c) w = word_max<F32>(w, m[i][c]);
      w = max16<F32>(w);
      const uint32_t s = scale_of(F32 ? w : max(first_of<F32>(w), second_of(w)));
      *reinterpret_cast<uint2*>(out + i * pitch) = t.v[i].bytes(value_of(s));
      if (cg == 0) scales[scale_place(rt * 8 + i)] = static_cast<uint8_t>(s);
    }
  }
  if (a.by_cols) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < W; ++c) {
      top[c] = word_max<F32>(top[c], static_cast<uint32_t>(__shfl_xor(static_cast<int>(top[c]), 16)));
      top[c] = word_max<F32>(top[c], static_cast<uint32_t>(__shfl_xor(static_cast<int>(top[c]), 32)));
      if ((threadIdx.x & 63) < 16) tops[wave][cg * W + c] = top[c];
    }
    __syncthreads();
    uint32_t scale[8];
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const int k = cg * W + c;
      const uint32_t w = word_max<F32>(word_max<F32>(tops[0][k], tops[1][k]), word_max<F32>(tops[2][k], tops[3][k]));
      scale[F32 ? c : 2 * c % 8] = scale_of(first_of<F32>(w));
      if (!F32) scale[(2 * c + 1) % 8] = scale_of(second_of(w));
    }
    if (rt == 0) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        a.col_scales[(static_cast<int64_t>(p) * a.col_blocks + kt) * kBlock + scale_place(cg * 8 + c)] = static_cast<uint8_t>(scale[c]);
    }
    const int64_t pitch = static_cast<int64_t>(a.g.blocks) * kBlock;
    write_columns<F32>(t, scale, lds, a.by_cols + static_cast<int64_t>(kt) * kBlock * pitch + static_cast<int64_t>(p) * kBlock, pitch, kBlock);
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(WeightArgs a) {
  constexpr int W = Tile<F32>::W;
  __shared__ __attribute__((aligned(16))) char lds[128 * 128];
  __shared__ uint32_t tops[4];
  const int ot = blockIdx.x, it = blockIdx.y, e = blockIdx.z;  // tiles of out, of in
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  const int col = ot * kBlock + cg * 8, n = min(8, max(0, a.out - col));
  const int ob = (a.out + kBlock - 1) / kBlock, ib = (a.in + kBlock - 1) / kBlock;
  Raw8<F32> raw[8];
  int have[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = it * kBlock + rt * 8 + i;
    have[i] = r < a.in ? n : 0;
    raw[i] = fetch8<F32>(a.w, e * a.expert_stride + r * a.ld, col, have[i]);
  }
  Tile<F32> t;
#pragma unroll
  for (int i = 0; i < 8; ++i) t.v[i] = Eight<F32>(settle8<F32>(raw[i], col, have[i]));
  uint32_t m[8][W], top[W];
  tile_magnitudes<F32>(t, m, top);
  uint32_t w = top[0];
#pragma unroll
  for (int c = 1; c < W; ++c) w = word_max<F32>(w, top[c]);
  w = max16<F32>(w);
  w = F32 ? w : max(first_of<F32>(w), second_of(w));
  w = max(w, static_cast<uint32_t>(__shfl_xor(static_cast<int>(w), 16)));
  w = max(w, static_cast<uint32_t>(__shfl_xor(static_cast<int>(w), 32)));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = w;
  __syncthreads();
  const uint32_t s = scale_of(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
  const int ib4 = (ib + 3) / 4 * 4, ob4 = (ob + 3) / 4 * 4;
  // a scale row's last tile also fills the places behind it, with 2^0
  if (threadIdx.x < 4) {
    const int i = static_cast<int>(threadIdx.x);
    if (i == 0 || (it == ib - 1 && it + i < ib4))
      a.forward_scales[(static_cast<int64_t>(e) * ob + ot) * ib4 + it + i] = static_cast<uint8_t>(i == 0 ? s : 127);
    if (a.backward && (i == 0 || (ot == ob - 1 && ot + i < ob4)))
      a.backward_scales[(static_cast<int64_t>(e) * ib + it) * ob4 + ot + i] = static_cast<uint8_t>(i == 0 ? s : 127);
  }
  if (a.backward) {
    const int64_t pitch = static_cast<int64_t>(ob) * kBlock;
    uint8_t* out = a.backward + (static_cast<int64_t>(e) * a.in + it * kBlock + rt * 8) * pitch + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (it * kBlock + rt * 8 + i < a.in) *reinterpret_cast<uint2*>(out + i * pitch) = t.v[i].bytes(value_of(s));
  }
  uint32_t scale[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) scale[c] = s;
  const int64_t pitch = static_cast<int64_t>(ib) * kBlock;
  write_columns<F32>(t, scale, lds, a.forward + (static_cast<int64_t>(e) * a.out + ot * kBlock) * pitch + it * kBlock, pitch, min(kBlock, a.out - ot * kBlock));
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  if (a.g.blocks == 0) return hipSuccess;
  const uint32_t grid = static_cast<uint32_t>(a.col_blocks) * static_cast<uint32_t>(a.g.blocks);
  if (a.f32)
    quantize_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    quantize_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(const WeightArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>((a.out + kBlock - 1) / kBlock), static_cast<uint32_t>((a.in + kBlock - 1) / kBlock),
                  static_cast<uint32_t>(a.experts));
  if (a.f32)
    quantize_weight_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    quantize_weight_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace she
