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
// 8192 x 8192 bf16 by rows and columns: 56 us, 4.8 TB/s (268 MB); 8192 x 2048 18;
// a weight of 2048 x 8192 both ways 16; five of 1001 x 2730 fp32 16, 5.1 TB/s.
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
// block, its first row and its rows. Every wave finds it by itself.
struct Found {
  int expert, block0, row0, rows;
};
__device__ __forceinline__ int blocks_of(int rows) { return rows > 0 ? (rows + kBlock - 1) / kBlock : 0; }
__device__ __forceinline__ Found find_group(const Groups& g, int p) {
  const int lane = threadIdx.x & 63, each = (g.experts + 63) / 64;
  const int from = min(lane * each, g.experts), to = min(from + each, g.experts);
  const int begin = group_row(g, from);
  int blocks = 0, lo = begin;
  for (int e = from; e < to; ++e) {
    const int hi = group_row(g, e + 1);
    blocks += blocks_of(hi - lo);
    lo = hi;
  }
  int pb = blocks;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(pb, d);
    if (lane >= d) pb += up;
  }
  const bool here = p >= pb - blocks && p < pb;
  pb -= blocks;
  lo = begin;
  Found f{-1, 0, 0, 0};
  for (int e = from; e < to; ++e) {
    const int hi = group_row(g, e + 1), b = blocks_of(hi - lo);
    if (p >= pb && p < pb + b) f = Found{e, pb, lo, hi - lo};
    pb += b;
    lo = hi;
  }
  const uint64_t found = __ballot(here);
  const int who = found ? __ffsll(static_cast<unsigned long long>(found)) - 1 : 0;
  f.expert = found ? __builtin_amdgcn_readlane(f.expert, who) : -1;
  f.block0 = __builtin_amdgcn_readlane(f.block0, who);
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

// ------------------------------------------------------------ the products' work
__device__ __forceinline__ uint32_t buffer_size(int64_t left) {
  return left <= 0 ? 0u : left > 0xfffffff0ll ? 0xfffffff0u : static_cast<uint32_t>(left);
}

// Each expert's first row tile and first block of padded rows; [experts]: all.
__device__ __forceinline__ void write_tables(const Groups& g, int per_tile, int* first_tile, int* first_block) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    const int each = (g.experts + 63) / 64, from = min(lane * each, g.experts), to = min(from + each, g.experts);
    int tiles = 0, blocks = 0, lo = group_row(g, from);
    const int begin = lo;
    for (int e = from; e < to; ++e) {
      const int hi = group_row(g, e + 1), b = blocks_of(hi - lo);
      blocks += b;
      tiles += (b + per_tile - 1) / per_tile;
      lo = hi;
    }
    int pt = tiles, pb = blocks;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int ut = __shfl_up(pt, d), ub = __shfl_up(pb, d);
      if (lane >= d) pt += ut, pb += ub;
    }
    pt -= tiles, pb -= blocks;
    lo = begin;
    for (int e = from; e < to; ++e) {
      const int hi = group_row(g, e + 1), b = blocks_of(hi - lo);
      first_tile[e] = pt;
      first_block[e] = min(pb, g.blocks);
      pb += b;
      pt += (b + per_tile - 1) / per_tile;
      lo = hi;
    }
    if (lane == 63) {
      first_tile[g.experts] = pt;
      first_block[g.experts] = min(pb, g.blocks);
    }
  }
  __syncthreads();
}

// Records of the products' work, one a thread. An XCD takes a contiguous range of a
// product's tiles, in groups of four row tiles, so that those in flight on one XCD
// share their operands in its L2. Experts have sums of different length: each XCD
// takes its part of every expert's tiles, another one for each (dW of eight experts of
// 16384 x 2048 x 2048 bf16: 88 us; with an expert an XCD 126). dW, the last product,
// goes by length, longest first, and the first product before the experts whose sums
// are shorter than its own: workgroups take the list to and fro, which then evens
// out (dx and dW of eight experts, three batches: 157, 142 and 145 us, in the experts'
// order 153, 160 and 164).
__device__ __forceinline__ void write_work(const Products& all, const Groups& g, int which, int* first_tile, int* first_block, int* order) {
  const int side = product_tile(static_cast<ProductTile>(all.tile)), per_tile = side / kBlock;
  if (g.offsets) write_tables(g, per_tile, first_tile, first_block);
  const ProductArgs& last = all.p[all.count > 0 ? all.count - 1 : 0];
  const uint32_t last_tiles = static_cast<uint32_t>((last.M + side - 1) / side) * ((last.N + side - 1) / side), last_per = (last_tiles + 7) / 8;
  const bool sorted = g.offsets && all.count > 0 && last.by_expert && last_tiles >= 16 && all.experts <= kThreads;
  uint32_t head = 0;  // experts in front of the first product
  if (sorted) {
    const int e = threadIdx.x;
    bool longer = false;
    if (e < all.experts) {
      const int mine = first_block[e + 1] - first_block[e];
      int rank = 0;
      for (int j = 0; j < all.experts; ++j) {
        const int its = first_block[j + 1] - first_block[j];
        rank += its > mine || (its == mine && j < e);
      }
      order[rank] = e;
      longer = all.count == 1 || mine > all.p[0].k_blocks;
    }
    head = static_cast<uint32_t>(__syncthreads_count(longer));
  }
  const int64_t record = static_cast<int64_t>(which) * kThreads + threadIdx.x;
  if (record >= 8ll * all.per) return;
  const uint32_t xcd = static_cast<uint32_t>(record / all.per);
  uint32_t n = static_cast<uint32_t>(record - static_cast<int64_t>(xcd) * all.per);
  WorkRecord w{};
  w.turns = kNoTileNorBehind;
  int q = 0;
  const bool front = sorted && n < head * last_per;
  if (front) q = all.count - 1;
  else if (sorted && all.count > 1) n -= head * last_per;
  for (; q < all.count; ++q) {
    const ProductArgs& p = all.p[q];
    const uint32_t tn = (p.N + side - 1) / side, experts = p.by_expert ? all.experts : 1;
    uint32_t tm = (p.M + side - 1) / side;
    int behind = 0;  // rows behind the last expert's
    if (!p.by_expert && g.offsets) {
      behind = g.n - group_row(g, g.experts);
      tm = first_tile[g.experts] + (behind + side - 1) / side;
    }
    const uint32_t tiles = tm * tn, per = (tiles + 7) / 8;  // of an XCD, of each expert
    const bool round = tiles < 16;                          // fewer than two of an expert an XCD: all experts' in turn
    const uint32_t length = round ? (tiles * experts + 7) / 8 : per * experts;
    if (sorted && all.count > 1 && q == 1 && !front) n += head * last_per;  // the experts behind the first product
    if (n >= length) {
      n -= length;
      continue;
    }
    w.turns = kNoTile;
    uint32_t expert, id;
    if (round) {
      const uint32_t at = n * 8 + xcd;
      if (at >= tiles * experts) break;
      expert = at / tiles;
      id = at - expert * tiles;
    } else {
      const uint32_t nth = n / per;
      id = (xcd + nth) % 8 * per + (n - nth * per);
      if (id >= tiles) break;
      expert = p.by_expert && sorted ? static_cast<uint32_t>(order[nth]) : nth;
    }
    const uint32_t group = id / (4 * tn), in_group = min(4u, tm - 4 * group);
    id -= group * 4 * tn;
    const int n0 = static_cast<int>(id / in_group) * side, trow = static_cast<int>(4 * group + id % in_group);
    int a_block = trow * per_tile, rows = min(side, p.M - trow * side), k0 = 0;
    int64_t c_row = static_cast<int64_t>(trow) * side;
    w.turns = p.k_blocks;
    if (p.by_expert) {
      if (g.offsets) {
        k0 = first_block[expert];
        w.turns = first_block[expert + 1] - k0;
      }
    } else if (g.offsets) {
      const int last = first_tile[g.experts];
      if (trow >= last) {
        const int down = (trow - last) * side;
        c_row = group_row(g, g.experts) + down;
        rows = min(side, behind - down);
        a_block = 0;
        w.turns = 0;
      } else {
        int lo = 0, hi = g.experts;  // the last expert whose first tile is not behind this one
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (first_tile[mid] <= trow) lo = mid;
          else hi = mid;
        }
        expert = static_cast<uint32_t>(lo);
        const int down = (trow - first_tile[lo]) * side, first_row = group_row(g, lo);
        c_row = first_row + down;
        rows = max(0, min(side, group_row(g, lo + 1) - first_row - down));
        a_block = first_block[lo] + (trow - first_tile[lo]) * per_tile;
      }
    }
    const int64_t a_at = static_cast<int64_t>(a_block) * kBlock * p.pitch + static_cast<int64_t>(k0) * kBlock;
    const int64_t b_at = n0 * p.pitch + static_cast<int64_t>(k0) * kBlock;
    const bool words = !p.by_expert;
    w.a = reinterpret_cast<uint64_t>(p.a) + a_at;
    w.b = reinterpret_cast<uint64_t>(p.b) + (words ? expert * p.b_stride : 0) + b_at;
    w.size_a = buffer_size(p.size_a - a_at);
    w.size_b = buffer_size(p.size_b - b_at);
    const int64_t a_step = static_cast<int64_t>(p.a_blocks) * kBlock, b_step = static_cast<int64_t>(p.b_blocks) * kBlock;
    const int64_t sa = k0 * a_step + static_cast<int64_t>(a_block) * kBlock;
    const int64_t sb = words ? static_cast<int64_t>(n0 / kBlock) * p.b_scale_pitch : k0 * b_step + n0;
    w.a_scales = reinterpret_cast<uint64_t>(p.a_scales) + sa;
    w.b_scales = reinterpret_cast<uint64_t>(p.b_scales) + (words ? expert * p.b_scale_stride : 0) + sb;
    w.a_scales_size = buffer_size(p.k_blocks * a_step - sa);
    w.b_scales_size = buffer_size((words ? static_cast<int64_t>(p.b_blocks) * p.b_scale_pitch : p.k_blocks * b_step) - sb);
    w.c = reinterpret_cast<uint64_t>(p.c) + ((p.by_expert ? expert * p.c_stride : 0) + c_row * p.ldc + n0) * (all.f32 ? 4 : 2);
    const uint32_t second = n0 / kBlock + 1 < p.b_blocks;
    w.shape = static_cast<uint32_t>(rows) | static_cast<uint32_t>(min(side, p.N - n0)) << 10 | static_cast<uint32_t>(words) << 20 | second << 21 |
              static_cast<uint32_t>(q) << 22;
    break;
  }
  all.work[record] = w;
}

constexpr int kMaxExperts = 1024;
constexpr int kTables = 2 * (kMaxExperts + 1) + kThreads, kLds = kBlock * kBlock;
static_assert(kLds >= 4 * kTables, "");

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a) {
  constexpr int W = Tile<F32>::W;
  __shared__ __attribute__((aligned(16))) char lds[kLds];
  __shared__ uint32_t tops[4][128];
  // the first workgroups write the records
  const uint32_t writers = (8 * static_cast<uint32_t>(a.products.per) + kThreads - 1) / kThreads;
  if (blockIdx.x < writers) {
    int* tables = reinterpret_cast<int*>(lds);
    write_work(a.products, a.g, static_cast<int>(blockIdx.x), tables, tables + kMaxExperts + 1, tables + 2 * (kMaxExperts + 1));
    return;
  }
  const uint32_t block = blockIdx.x - writers;
  const int p = static_cast<int>(block / a.col_blocks), kt = static_cast<int>(block - static_cast<uint32_t>(p) * a.col_blocks);
  const int cg = threadIdx.x & 15, rt = threadIdx.x >> 4;
  int row0 = p * kBlock, count = min(kBlock, a.g.n - row0);
  if (a.g.offsets) {
    const Found f = find_group(a.g, p);
    if (f.expert < 0) return;
    const int local = p - f.block0;
    row0 = f.row0 + local * kBlock;
    count = min(kBlock, f.rows - local * kBlock);
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

// Rows of x in 8 bits, each at the padded rows of all its slots: x is read once, where
// quantize_kernel would read it for every slot (2048 tokens x 8 slots x 2048 bf16:
// 13.2 us, 20). Tiles of 32 rows x 128 columns, so that there are enough of them.
constexpr int kScatterRows = 32;
template <bool F32>
__global__ __launch_bounds__(kThreads) void scatter_kernel(QuantizeArgs a) {
  constexpr int R = kScatterRows / 16;
  __shared__ int first_row[kMaxExperts + 1], first_block[kMaxExperts + 1], places[kScatterRows * kMaxScatter];
  const uint32_t writers = (8 * static_cast<uint32_t>(a.products.per) + kThreads - 1) / kThreads;
  if (blockIdx.x < writers) {
    write_work(a.products, a.g, static_cast<int>(blockIdx.x), first_row, first_block, places);
    return;
  }
  const uint32_t block = blockIdx.x - writers;
  const int rt = static_cast<int>(block / a.col_blocks), kt = static_cast<int>(block - static_cast<uint32_t>(rt) * a.col_blocks);
  const int row0 = rt * kScatterRows, count = min(kScatterRows, a.rows_in - row0), slots = static_cast<int>(a.slots);
  const int cg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int col = kt * kBlock + cg * 8, n = min(8, max(0, a.cols - col));
  Raw8<F32> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i] = fetch8<F32>(a.x, static_cast<int64_t>(row0 + r0 + 16 * i) * a.ld, col, r0 + 16 * i < count ? n : 0);
  constexpr int L = kScatterRows * kMaxScatter / kThreads;
  int rows[L];
#pragma unroll
  for (int k = 0; k < L; ++k) {
    const int i = threadIdx.x + k * kThreads;
    rows[k] = i < count * slots ? a.slot_rows[static_cast<int64_t>(row0) * slots + i] : -1;
  }
  // where each slot goes: its padded row, -1 for none
  write_tables(a.g, 1, first_row, first_block);
  for (int e = threadIdx.x; e <= a.g.experts; e += kThreads) first_row[e] = group_row(a.g, e);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < L; ++k) {
    const int r = rows[k];
    int place = -1;
    if (r >= 0 && r < first_row[a.g.experts]) {
      int lo = 0, hi = a.g.experts;  // the last expert whose first row is not behind r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first_row[mid] <= r) lo = mid;
        else hi = mid;
      }
      place = first_block[lo] * kBlock + r - first_row[lo];
      if (place < 0 || place >= a.g.blocks * kBlock) place = -1;
    }
    places[threadIdx.x + k * kThreads] = place;
  }
  __syncthreads();
  const int64_t pitch = static_cast<int64_t>(a.col_blocks) * kBlock;
  uint8_t* scales = a.row_scales + static_cast<int64_t>(kt) * a.g.blocks * kBlock;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + 16 * i;
    const Eight<F32> v(settle8<F32>(raw[i], col, r < count ? n : 0));
    uint32_t w = v.magnitude();
    w = max16<true>(w);
    const uint32_t s = scale_of(w);
    const uint2 bytes = v.bytes(value_of(s));
    if (r >= count) continue;
    for (int j = 0; j < slots; ++j) {
      const int place = places[r * slots + j];
      if (place < 0) continue;
      *reinterpret_cast<uint2*>(a.by_rows + place * pitch + col) = bytes;
      if (cg == 0) scales[(place & ~(kBlock - 1)) + scale_place(place & (kBlock - 1))] = static_cast<uint8_t>(s);
    }
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

int64_t work_length(const Products& a, int64_t rows, bool grouped) {
  const int64_t side = product_tile(static_cast<ProductTile>(a.tile));
  int64_t length = 0;
  for (int q = 0; q < a.count; ++q) {
    const ProductArgs& p = a.p[q];
    const int64_t tn = (p.N + side - 1) / side, used = a.experts < rows ? a.experts : rows;
    const int64_t tm = grouped && !p.by_expert ? (rows + (side - 1) * (used + 1)) / side : (p.M + side - 1) / side;
    const int64_t experts = p.by_expert ? a.experts : 1, tiles = tm * tn;
    // under 16 tiles all experts' go in turn; a grouped product may turn out to have so few
    const int64_t round = ((tiles < 16 ? tiles : 15) * experts + 7) / 8, parts = tiles < 16 ? 0 : (tiles + 7) / 8 * experts;
    length += round > parts ? round : parts;
  }
  return length;
}

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  const uint32_t writers = (8 * static_cast<uint32_t>(a.products.per) + kThreads - 1) / kThreads;
  const int tiles = a.slot_rows ? (a.rows_in + kScatterRows - 1) / kScatterRows : a.g.blocks;
  const int64_t all = static_cast<int64_t>(a.col_blocks) * tiles + writers;
  if (all == 0) return hipSuccess;
  // a launch has fewer than 2^32 threads; of so many tiles the values alone are 2^37 bytes and more
  if (all >= (int64_t(1) << 32) / kThreads) return hipErrorInvalidConfiguration;
  const uint32_t grid = static_cast<uint32_t>(all);
  if (a.slot_rows)
    a.f32 ? scatter_kernel<true><<<grid, kThreads, 0, s>>>(a) : scatter_kernel<false><<<grid, kThreads, 0, s>>>(a);
  else
    a.f32 ? quantize_kernel<true><<<grid, kThreads, 0, s>>>(a) : quantize_kernel<false><<<grid, kThreads, 0, s>>>(a);
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
