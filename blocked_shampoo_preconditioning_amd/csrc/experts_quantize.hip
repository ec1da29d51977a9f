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
// through LDS. Memory bounds it: 2 or 4 bytes in, 1 or 2 out an element.
#include "experts_device.h"

namespace she {

using shl::fetch8;
using shl::Raw8;
using shl::settle8;
using shl::unpack8;

namespace {

constexpr int kThreads = 256;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
  return max(v, o);
}
// The largest of 16 lanes, in all of them (rotations of a row of 16).
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = dpp_max<0x128>(v);
  v = dpp_max<0x124>(v);
  v = dpp_max<0x122>(v);
  return dpp_max<0x121>(v);
}

// The expert whose rows block p holds, by the first wave of a workgroup. Writes
// {expert, its first block, its first row tile, its first row, its rows}, -1 where
// p is behind all blocks; totals in sums (blocks, row tiles, rows).
struct Found {
  int32_t expert, block0, tile0, row0, rows;
  int32_t all_tiles, all_rows;
};
__device__ __forceinline__ void find_group(const Groups& g, int p, int tile_blocks, int32_t* first_block, Found* out) {
  const int lane = threadIdx.x & 63, each = (g.experts + 63) / 64;
  const int from = min(lane * each, g.experts), to = min(from + each, g.experts);
  auto row = [&](int e) { return group_row(g, e); };
  auto blocks_of = [&](int lo, int hi) { return hi > lo ? (hi - lo + kBlock - 1) / kBlock : 0; };
  int blocks = 0, tiles = 0;
  for (int e = from; e < to; ++e) {
    const int b = blocks_of(row(e), row(e + 1));
    blocks += b;
    tiles += (b + tile_blocks - 1) / tile_blocks;
  }
  int pb = blocks, pt = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int ub = __shfl_up(pb, d), ut = __shfl_up(pt, d);
    if (lane >= d) pb += ub, pt += ut;
  }
  if (lane == 63) {
    out->all_tiles = pt;
    out->all_rows = row(g.experts);
    if (first_block) first_block[g.experts] = min(pb, g.blocks);
    if (p >= pb) out->expert = -1;
  }
  pb -= blocks, pt -= tiles;
  for (int e = from; e < to; ++e) {
    const int lo = row(e), hi = row(e + 1), b = blocks_of(lo, hi);
    if (first_block) first_block[e] = min(pb, g.blocks);
    if (p >= pb && p < pb + b) {
      out->expert = e;
      out->block0 = pb;
      out->tile0 = pt;
      out->row0 = lo;
      out->rows = hi - lo;
    }
    pb += b;
    pt += (b + tile_blocks - 1) / tile_blocks;
  }
}

// A tile's eight rows and columns of a thread.
template <bool F32>
struct Tile {
  Raw8<F32> v[8];
};

// Columns: the tile's maxima by column are in `top` (four partial ones a
// column); the values go out transposed. `scales`: where the tile's 128 scales go.
template <bool F32>
__device__ __forceinline__ void write_columns(const Tile<F32>& t, const uint32_t (&scale)[8], char* lds, uint8_t* out, int64_t pitch, int rows) {
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  uint32_t w[8][2];
  float inv[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) inv[c] = inverse_of(scale[c]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r) unpack8<F32>(t.v[4 * h + r], x[r]);
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c][h] = pack4(x[0][c] * inv[c], x[1][c] * inv[c], x[2][c] * inv[c], x[3][c] * inv[c]);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int col = cg * 8 + c;
    uint32_t* q = reinterpret_cast<uint32_t*>(lds + col * 128 + (((rt >> 1) ^ (cg & 7)) << 4) + (rt & 1) * 8);
    q[0] = w[c][0];
    q[1] = w[c][1];
  }
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
  __shared__ __attribute__((aligned(16))) char lds[128 * 128];
  __shared__ uint32_t top[4][128];
  __shared__ Found found;
  const int p = static_cast<int>(blockIdx.x / a.col_blocks), kt = static_cast<int>(blockIdx.x - static_cast<uint32_t>(p) * a.col_blocks);
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  int row0 = p * kBlock, count = min(kBlock, a.g.n - row0);
  if (a.g.offsets) {
    const bool lead = kt == 0 && p == 0;
    if (threadIdx.x < 64) find_group(a.g, p, a.tile_blocks, lead ? a.first_block : nullptr, &found);
    __syncthreads();
    const Found f = found;
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
  Tile<F32> t;
  int64_t at[8];
  int have[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rt * 8 + i;
    have[i] = r < count ? n : 0;
    int64_t from = row0 + r;
    if (a.source && r < count) {
      const int32_t s = a.source[row0 + r];
      from = min(static_cast<uint32_t>(s < 0 ? ~s : s) / a.slots, static_cast<uint32_t>(a.rows_in - 1));
    }
    at[i] = from * a.ld;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) t.v[i] = fetch8<F32>(a.x, at[i], col, have[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) t.v[i] = settle8<F32>(t.v[i], col, have[i]);

  if (a.by_rows) {
    const int64_t pitch = static_cast<int64_t>(a.col_blocks) * kBlock;
    uint8_t* out = a.by_rows + (static_cast<int64_t>(p) * kBlock + rt * 8) * pitch + col;
    uint8_t* scales = a.row_scales + (static_cast<int64_t>(kt) * a.g.blocks + p) * kBlock;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8<F32>(t.v[i], x);
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = max(m, magnitude(x[q]));
      const uint32_t s = scale_of(max16(m));
      const float inv = inverse_of(s);
      const uint2 w = {pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv), pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
      *reinterpret_cast<uint2*>(out + i * pitch) = w;
      if (cg == 0) scales[scale_place(rt * 8 + i)] = static_cast<uint8_t>(s);
    }
  }
  if (a.by_cols) {
    uint32_t m[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) m[c] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8<F32>(t.v[i], x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[c] = max(m[c], magnitude(x[c]));
    }
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = max(m[c], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[c]), 16)));
      m[c] = max(m[c], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[c]), 32)));
      if ((threadIdx.x & 63) < 16) top[wave][cg * 8 + c] = m[c];
    }
    __syncthreads();
    uint32_t scale[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int k = cg * 8 + c;
      scale[c] = scale_of(max(max(top[0][k], top[1][k]), max(top[2][k], top[3][k])));
      if (rt == 0) a.col_scales[(static_cast<int64_t>(p) * a.col_blocks + kt) * kBlock + scale_place(k)] = static_cast<uint8_t>(scale[c]);
    }
    const int64_t pitch = static_cast<int64_t>(a.g.blocks) * kBlock;
    write_columns<F32>(t, scale, lds, a.by_cols + static_cast<int64_t>(kt) * kBlock * pitch + static_cast<int64_t>(p) * kBlock, pitch, kBlock);
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(WeightArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[128 * 128];
  __shared__ uint32_t top[4];
  const int ot = blockIdx.x, it = blockIdx.y, e = blockIdx.z;  // tiles of out, of in
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  const int col = ot * kBlock + cg * 8, n = min(8, max(0, a.out - col));
  const int ob = (a.out + kBlock - 1) / kBlock, ib = (a.in + kBlock - 1) / kBlock;
  Tile<F32> t;
  int have[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = it * kBlock + rt * 8 + i;
    have[i] = r < a.in ? n : 0;
    t.v[i] = fetch8<F32>(a.w, e * a.expert_stride + r * a.ld, col, have[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.v[i] = settle8<F32>(t.v[i], col, have[i]);
    float x[8];
    unpack8<F32>(t.v[i], x);
#pragma unroll
    for (int c = 0; c < 8; ++c) m = max(m, magnitude(x[c]));
  }
  m = max16(m);
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
  const uint32_t s = scale_of(max(max(top[0], top[1]), max(top[2], top[3])));
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
    const float inv = inverse_of(s);
    const int64_t pitch = static_cast<int64_t>(ob) * kBlock;
    uint8_t* out = a.backward + (static_cast<int64_t>(e) * a.in + it * kBlock + rt * 8) * pitch + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8<F32>(t.v[i], x);
      const uint2 w = {pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv), pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
      if (it * kBlock + rt * 8 + i < a.in) *reinterpret_cast<uint2*>(out + i * pitch) = w;
    }
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
