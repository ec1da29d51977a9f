// 8-bit products of up to 64 rows in all: the weights are read once, from memory
// into registers and the matrix cores, and x is quantized by every workgroup as it
// reads it, so that a call is one launch.
//
// The experts that have rows, one after the other, are the grid's second axis. A
// workgroup goes through tiles of 16 FN columns of one matrix, every gridDim.x-th.
// Its waves take K blocks in turn, keep the 8 bits of theirs of x (up to KEEP
// blocks a wave) over all tiles, and have the next tile's weights on their way
// while one is multiplied; a tile's sums are joined through LDS in the order of the
// waves. More than 16 rows are taken 16 at a time, the weights from the caches
// again.
//
// What bounds it are the weights' bytes (32 rows of eight experts of 2048 x 8192: 29
// to 30 us, 4.5 TB/s), for a single token the launch and the chain of loads, join and
// store (2048 x 8192: 7.1 us). Above 16 rows of one matrix it is the number of times that
// the weights come from the caches.
#include <type_traits>

#include "experts_device.h"

namespace she {

using shl::fetch8;
using shl::floatx4;
using shl::Raw8;
using shl::settle8;

namespace {

// The expert that is the s-th of those with rows: its number, first row and rows;
// count 0 if there is none. Every wave finds it by itself.
struct Chosen {
  int expert, row0, count, all_rows;
};
__device__ __forceinline__ Chosen find_expert(const Groups& g, int s) {
  const int lane = threadIdx.x & 63, each = (g.experts + 63) / 64;
  const int from = min(lane * each, g.experts), to = min(from + each, g.experts);
  int have = 0, lo = group_row(g, from);
  const int begin = lo;
  for (int e = from; e < to; ++e) {
    const int hi = group_row(g, e + 1);
    have += hi > lo;
    lo = hi;
  }
  const int all_rows = __shfl(lo, 63);
  int upto = have;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(upto, d);
    if (lane >= d) upto += up;
  }
  int at = upto - have, expert = 0, row0 = 0, count = 0;
  const bool here = s >= at && s < upto;
  lo = begin;
  for (int e = from; here && e < to; ++e) {
    const int hi = group_row(g, e + 1);
    if (hi > lo && at++ == s) expert = e, row0 = lo, count = min(hi - lo, kFewRows);
    lo = hi;
  }
  const uint64_t found = __ballot(here);
  const int who = found ? __ffsll(static_cast<unsigned long long>(found)) - 1 : 0;
  return Chosen{__builtin_amdgcn_readlane(expert, who), __builtin_amdgcn_readlane(row0, who), __builtin_amdgcn_readlane(count, who), all_rows};
}

// KEEP: K blocks a wave may have; 0: any number, for one tile a workgroup.
template <bool F32, int FN, int NW, int KEEP>
__global__ __launch_bounds__(64 * NW, 2) void few_kernel(FewArgs a) {
  constexpr int COLS = 16 * FN, PITCH = COLS + 4, BUFFERS = KEEP ? KEEP : 2;
  __shared__ __attribute__((aligned(16))) float sums[2][NW * 16 * PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  int expert = 0, row0 = 0, count = a.g.n;
  const int tiles = (a.N + COLS - 1) / COLS;
  if (a.g.offsets) {
    const Chosen c = find_expert(a.g, blockIdx.y);
    expert = c.expert, row0 = c.row0, count = c.count;
    if (blockIdx.y == 0) {  // rows behind the last expert's
      for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x)
        for (int i = threadIdx.x; i < (a.g.n - c.all_rows) * COLS; i += 64 * NW) {
          const int col = tile * COLS + i % COLS;
          const int64_t at = static_cast<int64_t>(c.all_rows + i / COLS) * a.ldc + col;
          if (col < a.N) {
            if (F32)
              static_cast<float*>(a.c)[at] = 0.f;
            else
              static_cast<uint16_t*>(a.c)[at] = 0;
          }
        }
    }
    if (count == 0) return;
  }
  const int blocks = (a.K + kBlock - 1) / kBlock;
  const uint8_t* weights = a.b + expert * a.b_stride;
  const uint8_t* scales = a.b_scales + expert * a.b_scale_stride;

  // Of a K block a lane has 32 values of one row of x and of each operand of the
  // weights: 16 from 16 q4 on and 16 from 64 + 16 q4 on.
  struct Weights {
    int4v w[FN][2];
    uint32_t scale;
  };
  struct Row {
    Raw8<F32> x[4];
  };
  struct Bytes {
    int8v b;
    uint32_t scale;
  };
  auto load_w = [&](int tile, int kb, Weights& s) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const uint8_t* w = weights + static_cast<int64_t>(min(tile * COLS + 16 * j + r16, a.N - 1)) * a.pitch_b + kb * kBlock + 16 * q4;
      s.w[j][0] = *reinterpret_cast<const int4v*>(w);
      s.w[j][1] = *reinterpret_cast<const int4v*>(w + 64);
    }
    s.scale = *reinterpret_cast<const uint32_t*>(scales + static_cast<int64_t>(tile * COLS / kBlock) * a.b_scale_pitch + (kb & ~3)) >> (kb & 3) * 8 & 255u;
  };
  auto column = [&](int kb, int c) { return kb * kBlock + (c >> 1) * 64 + q4 * 16 + (c & 1) * 8; };
  auto load_x = [&](int kb, int64_t at, Row& row) {
#pragma unroll
    for (int c = 0; c < 4; ++c) row.x[c] = fetch8<F32>(a.x, at, column(kb, c), min(8, max(0, a.K - column(kb, c))));
  };
  auto quantize = [&](int kb, const Row& row) {
    Eight<F32> v[4];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[c] = Eight<F32>(settle8<F32>(row.x[c], column(kb, c), min(8, max(0, a.K - column(kb, c)))));
      top = max(top, v[c].magnitude());
    }
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
    Bytes r;
    r.scale = scale_of(top);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint2 w = v[c].bytes(value_of(r.scale));
      r.b[2 * c] = static_cast<int>(w.x);
      r.b[2 * c + 1] = static_cast<int>(w.y);
    }
    return r;
  };
  floatx4 acc[FN];
  auto multiply = [&](const Bytes& x, const Weights& s) {
    if constexpr (F32) {
      const float sx = value_of(x.scale), sw = value_of(s.scale);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8 u;
        widen(x.b[2 * k], sx, u, 0);
        widen(x.b[2 * k + 1], sx, u, 4);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          bf16x8 y;
          widen(s.w[j][k >> 1][2 * (k & 1)], sw, y, 0);
          widen(s.w[j][k >> 1][2 * (k & 1) + 1], sw, y, 4);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, u, acc[j], 0, 0, 0);
        }
      }
    } else {
      const int sw = static_cast<int>(s.scale);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int8v y = __builtin_shufflevector(s.w[j][0], s.w[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x.b, acc[j], 0, 0, 0, sw, 0, static_cast<int>(x.scale));
      }
    }
  };

  int buf = 0;
  for (int first = 0; first < count; first += 16) {
    // weights first, since x's loads wait for the row's number
    int tile = blockIdx.x;
    Weights w[BUFFERS];
#pragma unroll
    for (int s = 0; s < BUFFERS; ++s)
      if (wave + s * NW < blocks) load_w(tile, wave + s * NW, w[s]);
    const int r = row0 + min(first + r16, count - 1);
    int64_t from = r;
    if (a.source) {
      const int32_t src = a.source[r];
      from = min(static_cast<uint32_t>(src < 0 ? ~src : src) / a.slots, static_cast<uint32_t>(a.rows_in - 1));
    }
    const int64_t x_at = from * a.ld_x;
    Row row;
    Bytes x[BUFFERS];
    if (wave < blocks) load_x(wave, x_at, row);
    if (KEEP) {
#pragma unroll
      for (int s = 0; s < BUFFERS; ++s) {
        const int kb = wave + s * NW;
        if (kb >= blocks) continue;
        const Row now = row;
        if (s + 1 < BUFFERS && kb + NW < blocks) load_x(kb + NW, x_at, row);
        x[s] = quantize(kb, now);
      }
    }
    for (; tile < tiles; tile += gridDim.x) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (KEEP) {
        const int next = tile + static_cast<int>(gridDim.x);
#pragma unroll
        for (int s = 0; s < BUFFERS; ++s) {
          const int kb = wave + s * NW;
          if (kb >= blocks) continue;
          multiply(x[s], w[s]);
          if (next < tiles) load_w(next, kb, w[s]);
        }
      } else {
        for (int kb0 = wave; kb0 < blocks; kb0 += 2 * NW) {
#pragma unroll
          for (int s = 0; s < BUFFERS; ++s) {
            const int kb = kb0 + s * NW;
            if (kb >= blocks) continue;
            const Bytes now = quantize(kb, row);
            if (kb + NW < blocks) load_x(kb + NW, x_at, row);
            multiply(now, w[s]);
            if (kb + 2 * NW < blocks) load_w(tile, kb + 2 * NW, w[s]);
          }
        }
      }
      // a lane has row r16 and columns 16 j + 4 q4 + 0..3. Two buffers in turn: the
      // one that is written was read two tiles ago, before the last barrier. Global
      // loads go on over it.
      float* mine = sums[buf] + wave * (16 * PITCH);
#pragma unroll
      for (int j = 0; j < FN; ++j) *reinterpret_cast<floatx4*>(mine + r16 * PITCH + 16 * j + 4 * q4) = acc[j];
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const int rows = min(16, count - first);
      for (int i = threadIdx.x; i < rows * COLS; i += 64 * NW) {
        const int r = i / COLS, c = i % COLS, col = tile * COLS + c;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) v += sums[buf][k * (16 * PITCH) + r * PITCH + c];
        if (col < a.N) {
          const int64_t at = static_cast<int64_t>(row0 + first + r) * a.ldc + col;
          if (F32)
            static_cast<float*>(a.c)[at] = v;
          else
            static_cast<uint16_t*>(a.c)[at] = shl::f32_to_bf16(v);
        }
      }
      buf ^= 1;
    }
  }
}

template <bool F32>
void start(const FewArgs& a, hipStream_t s) {
  constexpr int NW = 8, KEEP = F32 ? 2 : 4;  // as registers allow
  const int64_t experts = a.g.offsets ? min(a.g.experts, a.g.n) : 1;
  // Tiles of 32 columns where that leaves each CU one, else of 16. Where there are
  // more than two for each CU, one workgroup a CU goes through them with x kept (32
  // rows of 8 experts of 2048 x 8192: 29 us, two a CU 36, four 44, a workgroup for
  // each tile 62; one token of 2048 x 8192, one tile a CU: 7.1, with x kept 9.2).
  const bool wide = experts * a.N >= 32 * 256;
  const int64_t tiles = (a.N + (wide ? 31 : 15)) / (wide ? 32 : 16), most = (256 + experts - 1) / experts;
  const bool keep = tiles > 2 * most && (a.K + kBlock - 1) / kBlock <= KEEP * NW;
  const dim3 grid(static_cast<uint32_t>(keep ? most : tiles), static_cast<uint32_t>(experts));
  if (keep)  // tiles of 16 are never more than two a CU
    few_kernel<F32, 2, NW, KEEP><<<grid, 64 * NW, 0, s>>>(a);
  else if (wide)
    few_kernel<F32, 2, NW, 0><<<grid, 64 * NW, 0, s>>>(a);
  else
    few_kernel<F32, 1, NW, 0><<<grid, 64 * NW, 0, s>>>(a);
}

}  // namespace

hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  if (a.g.n == 0) return hipSuccess;
  a.f32 ? start<true>(a, s) : start<false>(a, s);
  return hipGetLastError();
}

}  // namespace she
