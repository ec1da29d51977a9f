// Tokens sorted by expert and back.
//
// The sort is a stable counting sort: ranks among equal ids are counted in a
// wave by ballots over the bits of an id, across waves and workgroups by sums of
// counts in a fixed order, so nothing goes by the order of atomics. The copies
// go by token: a token's row is read once for all its slots, and since a slot
// that is left out has a row too, behind the experts', every row is written by
// exactly one slot and none needs clearing first.
//
// Memory bounds the copies, a few launches' length the sort: 16384 tokens x 8 x 2048
// bf16 sort 4.8 and 7.0 us, dispatch 117 (604 MB, 5.2 TB/s), combine 117 to 122 (5.0 to
// 5.2 TB/s), its gradient 233 (1.14 GB, 4.9 TB/s); of a single token every kernel takes
// 2.5 to 3.3.
#include "experts_kernels.h"
#include "layer_device.h"

namespace she {

using shl::fetch8;
using shl::Raw8;
using shl::settle8;
using shl::store8;
using shl::uint4v;
using shl::unpack8;

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr uint32_t kMaxExperts = 1024;

// The id of a slot, `experts` for one that is left out.
__device__ __forceinline__ uint32_t slot_expert(const SortArgs& a, uint32_t slot) {
  const uint32_t t = slot / a.slots, j = slot - t * a.slots;
  const int64_t at = t * a.ld_ids + j;
  const int64_t id = a.wide ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
  return id >= 0 && id < static_cast<int64_t>(a.experts) ? static_cast<uint32_t>(id) : a.experts;
}

// The lanes of this wave with the same value (of `bits` bits) as this lane's.
__device__ __forceinline__ uint64_t same_lanes(uint32_t v, int bits, bool on) {
  uint64_t m = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const bool bit = v >> b & 1;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

// Each wave's slots: a contiguous part of the workgroup's, in order.
__device__ __forceinline__ void wave_range(const SortArgs& a, uint32_t& first, uint32_t& last) {
  const uint32_t each = (a.per_block / kSortWaves + 63) / 64 * 64;
  const uint64_t from = static_cast<uint64_t>(blockIdx.x) * a.per_block, wave = threadIdx.x >> 6;
  const uint64_t end = min(from + a.per_block, static_cast<uint64_t>(a.total));
  first = static_cast<uint32_t>(min(from + wave * each, end));
  last = static_cast<uint32_t>(min(from + (wave + 1) * each, end));
}

// Counts of each expert (and of slots left out) by wave, into count[wave][e]. Up to
// 64 KEEP slots of a wave are read at once and kept.
template <int KEEP>
__device__ __forceinline__ void count_waves(const SortArgs& a, uint32_t* count, uint32_t (&kept)[KEEP > 0 ? KEEP : 1]) {
  const uint32_t n = a.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t first, last;
  wave_range(a, first, last);
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const uint32_t slot = first + 64 * k + lane;
    kept[k] = slot < last ? slot_expert(a, slot) : 0;
  }
  for (uint32_t i = threadIdx.x; i < n * kSortWaves; i += kSortThreads) count[i] = 0;
  __syncthreads();
  if (KEEP) {
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (first + 64 * k + lane < last) atomicAdd(&count[wave * n + kept[k]], 1u);
  } else {
    for (uint32_t i = first; i < last; i += 64)
      if (i + lane < last) atomicAdd(&count[wave * n + slot_expert(a, i + lane)], 1u);
  }
  __syncthreads();
}

// Sort, first of two launches: the counts of each workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t count[kSortWaves * (kMaxExperts + 1)];
  uint32_t none[1];
  count_waves<0>(a, count, none);
  const uint32_t n = a.experts + 1;
  for (uint32_t e = threadIdx.x; e < n; e += kSortThreads) {
    uint32_t sum = 0;
    for (int w = 0; w < kSortWaves; ++w) sum += count[w * n + e];
    a.counts[static_cast<int64_t>(blockIdx.x) * n + e] = sum;
  }
}

// Sort, second launch, or the only one where one workgroup does all: places.
// 131072 slots of 64 experts: 128 workgroups; one token: what a launch costs.
template <int KEEP>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ uint32_t count[kSortWaves * (kMaxExperts + 1)];
  __shared__ uint32_t before[kMaxExperts + 1], all[kMaxExperts + 1], wave_sum[kSortWaves];
  const uint32_t n = a.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // counts of the workgroups before this one, and of all: several threads an
  // expert, each with every parts-th workgroup
  for (uint32_t e = threadIdx.x; e < n; e += kSortThreads) before[e] = all[e] = 0;
  uint32_t kept[KEEP > 0 ? KEEP : 1];
  count_waves<KEEP>(a, count, kept);
  if (a.blocks > 1) {
    const uint32_t parts = max(1u, kSortThreads / n);
    for (uint32_t i = threadIdx.x; i < n * parts; i += kSortThreads) {
      const uint32_t part = i / n, e = i - part * n;
      uint32_t b = 0, s = 0;
#pragma unroll 8
      for (uint32_t k = part; k < a.blocks; k += parts) {
        const uint32_t c = a.counts[static_cast<int64_t>(k) * n + e];
        b += k < blockIdx.x ? c : 0;
        s += c;
      }
      atomicAdd(&before[e], b);
      atomicAdd(&all[e], s);
    }
    __syncthreads();
  } else {
    for (uint32_t e = threadIdx.x; e < n; e += kSortThreads) {
      uint32_t s = 0;
      for (int w = 0; w < kSortWaves; ++w) s += count[w * n + e];
      all[e] = s;
    }
    __syncthreads();
  }
  // exclusive sums over the experts; thread i has experts i and, where there are
  // 1025 counts, the last of them comes behind all others
  const uint32_t mine = threadIdx.x < n ? all[threadIdx.x] : 0;
  uint32_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(sum, d);
    if (lane >= static_cast<uint32_t>(d)) sum += up;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  uint32_t lower = 0, total = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    lower += w < static_cast<int>(wave) ? wave_sum[w] : 0;
    total += wave_sum[w];
  }
  sum += lower - mine;
  auto place = [&](uint32_t e, uint32_t start) {
    if (blockIdx.x == 0) a.offsets[e] = static_cast<int32_t>(start);
    uint32_t at = start + before[e];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = count[w * n + e];
      count[w * n + e] = at;
      at += c;
    }
  };
  if (threadIdx.x < n) place(threadIdx.x, sum);
  if (threadIdx.x == 0 && n > kSortThreads) place(kSortThreads, total);
  __syncthreads();
  // every wave goes through its slots again, 64 at a time
  uint32_t first, last;
  wave_range(a, first, last);
  const int bits = 32 - __clz(a.experts);
  uint32_t* next = count + wave * n;
  auto set_places = [&](uint32_t slot, uint32_t e) {
    const bool on = slot < last;
    const uint64_t same = same_lanes(e, bits, on);
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    uint32_t r = 0;
    if (on) r = next[e] + rank;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) next[e] = r + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (on) {
      const bool in = e < a.experts;
      a.rows[slot] = static_cast<int32_t>(in ? r : ~r);
      a.source[r] = static_cast<int32_t>(in ? slot : ~slot);
    }
  };
  if (KEEP) {
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (first + 64 * k < last) set_places(first + 64 * k + lane, kept[k]);
  } else {
    for (uint32_t i = first; i < last; i += 64) set_places(i + lane, i + lane < last ? slot_expert(a, i + lane) : 0);
  }
}

// ------------------------------------------------------------------ routes
template <bool F32>
__device__ __forceinline__ Raw8<F32> zeros8() {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.w[i] = uint4v{0, 0, 0, 0};
  return r;
}

// Eight elements as they are, or a row's last n < 8. Sorted rows are written past
// the caches (non-temporal): kept there, they are written back while the next
// kernel reads. All of a training pass of 8192 tokens x 2 x 2048 bf16 107 -> 89 us,
// of 16384 x 8 x 2048 612 -> 590 (dispatch alone 90 -> 120, each combine 146 -> 118).
// Only rows of whole cache lines are (`past`): 3001 x 3 x 777 fp32 10.2 us, so 12.3.
template <bool F32>
__device__ __forceinline__ void store_raw8(void* p, int64_t off, int n, const Raw8<F32>& r, bool past) {
  if (n == 8) {
    char* q = static_cast<char*>(p) + off * (F32 ? 4 : 2);
    if (past) {
      __builtin_nontemporal_store(r.w[0], reinterpret_cast<uint4v*>(q));
      if (F32) __builtin_nontemporal_store(r.w[F32 ? 1 : 0], reinterpret_cast<uint4v*>(q + 16));
    } else {
      __builtin_memcpy(q, &r.w[0], 16);
      if (F32) __builtin_memcpy(q + 16, &r.w[F32 ? 1 : 0], 16);
    }
  } else {
    constexpr int W = F32 ? 8 : 4;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = r.w[i / 4][i % 4];
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      if (F32)
        static_cast<uint32_t*>(p)[off + k] = w[0];
      else
        static_cast<uint16_t*>(p)[off + k] = static_cast<uint16_t>(w[0]);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t up = i + 1 < W ? w[i + 1 < W ? i + 1 : 0] : 0u;
        w[i] = F32 ? up : w[i] >> 16 | up << 16;
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ Raw8<F32> pack8(const float (&v)[8]) {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 8 : 4); ++i) r.w[i / 4][i % 4] = F32 ? __float_as_uint(v[i]) : shl::pack_bf16(v[2 * i % 8], v[(2 * i + 1) % 8]);
  return r;
}

// A slot's row: `kept` if it takes part, `row` < total if it has one at all.
struct Slot {
  uint32_t row;
  bool kept, any;
};
__device__ __forceinline__ Slot read_slot(const RouteArgs& a, uint32_t slot) {
  const int32_t r = a.rows[slot];
  Slot s;
  s.row = static_cast<uint32_t>(r < 0 ? ~r : r);
  s.any = s.row < a.total;
  s.kept = r >= 0 && s.any;
  return s;
}

// A wave takes a token (grid x) and NC groups of 512 columns of it (grid y), in
// NC groups of eight a lane.
template <int NC>
struct Columns {
  int col[NC], n[NC];
  __device__ __forceinline__ Columns(int width, int first, int step) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      col[c] = first + c * step;
      n[c] = min(8, max(0, width - col[c]));
    }
  }
};

constexpr int kRouteWaves = 4;

template <bool F32, int NC>
__global__ __launch_bounds__(64 * kRouteWaves) void dispatch_kernel(RouteArgs a) {
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (token >= a.tokens) return;
  const Columns<NC> c(a.width, static_cast<int>(blockIdx.y * (NC * 512) + (threadIdx.x & 63) * 8), 512);
  Raw8<F32> v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] = fetch8<F32>(a.x, token * a.ld_x, c.col[i], c.n[i]);
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] = settle8<F32>(v[i], c.col[i], c.n[i]);
  const uint32_t first = static_cast<uint32_t>(token) * a.slots;
  for (uint32_t j = 0; j < a.slots; ++j) {
    const Slot s = read_slot(a, first + j);
    if (!s.any) continue;
    const int64_t at = static_cast<int64_t>(s.row) * a.ld_xs;
#pragma unroll
    for (int i = 0; i < NC; ++i) store_raw8<F32>(a.xs, at + c.col[i], c.n[i], s.kept ? v[i] : zeros8<F32>(), a.past);
  }
}

template <bool F32, int NC>
__global__ __launch_bounds__(64 * kRouteWaves) void combine_kernel(RouteArgs a) {
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (token >= a.tokens) return;
  const Columns<NC> c(a.width, static_cast<int>(blockIdx.y * (NC * 512) + (threadIdx.x & 63) * 8), 512);
  const uint32_t first = static_cast<uint32_t>(token) * a.slots;
  float sum[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[i][q] = 0.f;
  // four slots' rows on their way at once
  for (uint32_t j0 = 0; j0 < a.slots; j0 += 4) {
    Raw8<F32> v[4][NC];
    float w[4];
    bool kept[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      kept[k] = false;
      if (j0 + k >= a.slots) continue;
      const Slot s = read_slot(a, first + j0 + k);
      kept[k] = s.kept;
      if (!s.kept) continue;
      w[k] = a.weights ? a.weights[first + j0 + k] : 1.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) v[k][i] = fetch8<F32>(a.ys, static_cast<int64_t>(s.row) * a.ld_ys, c.col[i], c.n[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!kept[k]) continue;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float x[8];
        unpack8<F32>(settle8<F32>(v[k][i], c.col[i], c.n[i]), x);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[i][q] = fmaf(w[k], x[q], sum[i][q]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) store8(a.y, token * a.ld_y + c.col[i], c.n[i], F32, sum[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// W waves a token; each pass over the row has NC groups of eight a lane.
template <bool F32, int NC, int W>
__global__ __launch_bounds__(64 * kRouteWaves) void combine_backward_kernel(RouteArgs a) {
  __shared__ float part[2][kRouteWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t token = W == 1 ? static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave : static_cast<int64_t>(blockIdx.x);
  if (token >= a.tokens) return;
  constexpr int STEP = 512 * W, PASS = NC * STEP;
  const int lane8 = ((W == 1 ? 0 : wave * 64) + lane) * 8;
  const uint32_t first = static_cast<uint32_t>(token) * a.slots;
  const bool one = a.width <= PASS;
  Raw8<F32> dy[NC];
  auto load_dy = [&](const Columns<NC>& c) {
#pragma unroll
    for (int i = 0; i < NC; ++i) dy[i] = fetch8<F32>(a.x, token * a.ld_x, c.col[i], c.n[i]);
#pragma unroll
    for (int i = 0; i < NC; ++i) dy[i] = settle8<F32>(dy[i], c.col[i], c.n[i]);
  };
  const Columns<NC> c0(a.width, lane8, STEP);
  Raw8<F32> next[NC];
  auto load_ys = [&](const Slot& s, const Columns<NC>& c) {
#pragma unroll
    for (int i = 0; i < NC; ++i) next[i] = s.kept ? fetch8<F32>(a.ys, static_cast<int64_t>(s.row) * a.ld_ys, c.col[i], c.n[i]) : zeros8<F32>();
  };
  Slot s = read_slot(a, first);
  load_ys(s, c0);
  if (one) load_dy(c0);
  for (uint32_t j = 0; j < a.slots; ++j) {
    const Slot at = s;
    const float w = at.kept ? a.weights[first + j] : 0.f;
    float dot = 0.f;
    for (int col0 = 0; col0 < a.width; col0 += PASS) {
      const Columns<NC> c(a.width, col0 + lane8, STEP);
      if (!one) load_dy(c);
      Raw8<F32> ys[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) ys[i] = at.kept ? settle8<F32>(next[i], c.col[i], c.n[i]) : next[i];
      // what comes next is loaded before this is stored: a load waits for the stores before it
      if (col0 + PASS < a.width) {
        load_ys(at, Columns<NC>(a.width, col0 + PASS + lane8, STEP));
      } else if (j + 1 < a.slots) {
        s = read_slot(a, first + j + 1);
        load_ys(s, c0);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float g[8], v[8];
        unpack8<F32>(dy[i], g);
        unpack8<F32>(ys[i], v);
        if (at.kept) {
#pragma unroll
          for (int q = 0; q < 8; ++q) dot = fmaf(g[q], v[q], dot);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) g[q] = at.kept ? g[q] * w : 0.f;
        if (at.any) store_raw8<F32>(a.xs, static_cast<int64_t>(at.row) * a.ld_xs + c.col[i], c.n[i], pack8<F32>(g), a.past);
      }
    }
    dot = wave_sum(dot);
    if (W > 1) {
      if (lane == 0) part[j & 1][wave] = dot;
      __syncthreads();
      dot = 0.f;
#pragma unroll
      for (int i = 0; i < kRouteWaves; ++i) dot += part[j & 1][i];
    }
    if (lane == 0 && (W == 1 || wave == 0)) a.dweights[first + j] = dot;
  }
}

// Groups of 512 columns of a wave: as many as leave some thousand waves.
int columns_per_wave(const RouteArgs& a) {
  const int64_t groups = (a.width + 511) / 512;
  if (groups >= 4 && a.tokens * ((groups + 3) / 4) >= 4096) return 4;
  return groups >= 2 && a.tokens * ((groups + 1) / 2) >= 4096 ? 2 : 1;
}

// A launch has fewer than 2^32 threads: at most this many tokens each.
constexpr int64_t kTokensALaunch = int64_t(1) << 23;
template <class F>
hipError_t in_parts(const RouteArgs& a, F&& f) {
  const int64_t e = a.f32 ? 4 : 2;
  for (int64_t t = 0; t < a.tokens; t += kTokensALaunch) {
    RouteArgs part = a;
    part.tokens = min(a.tokens - t, kTokensALaunch);
    part.rows = a.rows + t * a.slots;
    if (a.weights) part.weights = a.weights + t * a.slots;
    if (a.dweights) part.dweights = a.dweights + t * a.slots;
    if (a.x) part.x = static_cast<const char*>(a.x) + t * a.ld_x * e;
    if (a.y) part.y = static_cast<char*>(a.y) + t * a.ld_y * e;
    const hipError_t err = f(part);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <class F>
hipError_t by_columns(const RouteArgs& a, F&& f) {
  if (a.width == 0) return hipSuccess;
  const int nc = columns_per_wave(a);
  const dim3 grid(static_cast<uint32_t>((a.tokens + kRouteWaves - 1) / kRouteWaves), static_cast<uint32_t>((a.width + 512 * nc - 1) / (512 * nc)));
  if (nc == 4)
    f(std::integral_constant<int, 4>{}, grid);
  else if (nc == 2)
    f(std::integral_constant<int, 2>{}, grid);
  else
    f(std::integral_constant<int, 1>{}, grid);
  return hipGetLastError();
}

}  // namespace

void sort_plan(int64_t total, uint32_t& blocks, uint32_t& per_block) {
  // One workgroup up to 4096 slots (one launch and two, us: 2048 slots of 2 to 256
  // experts 4.8 to 5.5 and 6.5 to 7.3, 4096 6.2 to 7.2 and 6.6 to 7.5, 8192 11 to 14 and
  // 6.9 to 8.2; of 1024 experts 4096 8.6 and 10, 8192 16 and 12);
  // then at least 1024 of them a workgroup, and at most 256 workgroups, whose counts
  // each of them sums.
  const int64_t each = total <= 4096 ? total : (total + 255) / 256;
  per_block = static_cast<uint32_t>((each > 0 ? each + 1023 : 1024) / 1024 * 1024);
  blocks = static_cast<uint32_t>((total + per_block - 1) / per_block);
  if (blocks == 0) blocks = 1;
}

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
  if (a.blocks > 1) sort_count_kernel<<<a.blocks, kSortThreads, 0, s>>>(a);
  if (a.per_block <= 1024)
    sort_place_kernel<1><<<a.blocks, kSortThreads, 0, s>>>(a);
  else if (a.per_block <= 4096)
    sort_place_kernel<4><<<a.blocks, kSortThreads, 0, s>>>(a);
  else
    sort_place_kernel<0><<<a.blocks, kSortThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const RouteArgs& all, hipStream_t s) {
  return in_parts(all, [&](const RouteArgs& a) {
    return by_columns(a, [&](auto nc, dim3 grid) {
      if (a.f32)
        dispatch_kernel<true, decltype(nc)::value><<<grid, 64 * kRouteWaves, 0, s>>>(a);
      else
        dispatch_kernel<false, decltype(nc)::value><<<grid, 64 * kRouteWaves, 0, s>>>(a);
    });
  });
}

hipError_t launch_combine(const RouteArgs& all, hipStream_t s) {
  return in_parts(all, [&](const RouteArgs& a) {
    return by_columns(a, [&](auto nc, dim3 grid) {
      if (a.f32)
        combine_kernel<true, decltype(nc)::value><<<grid, 64 * kRouteWaves, 0, s>>>(a);
      else
        combine_kernel<false, decltype(nc)::value><<<grid, 64 * kRouteWaves, 0, s>>>(a);
    });
  });
}

static hipError_t launch_combine_backward_part(const RouteArgs& a, hipStream_t s) {
  auto start = [&](auto nc, auto w) {
    constexpr int NC = decltype(nc)::value, W = decltype(w)::value;
    const uint32_t grid = static_cast<uint32_t>(W == 1 ? (a.tokens + kRouteWaves - 1) / kRouteWaves : a.tokens);
    if (a.f32)
      combine_backward_kernel<true, NC, W><<<grid, 64 * kRouteWaves, 0, s>>>(a);
    else
      combine_backward_kernel<false, NC, W><<<grid, 64 * kRouteWaves, 0, s>>>(a);
  };
  using std::integral_constant;
  // one wave a token where a pass of it holds the row and there are some thousand;
  // else four (3001 tokens x 3 x 777 fp32: 18.4 us with four, 12.4 with one)
  if (a.width <= 2048 && a.tokens >= 1024) {
    if (a.width <= 512)
      start(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (a.width <= 1024)
      start(integral_constant<int, 2>{}, integral_constant<int, 1>{});
    else
      start(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  } else if (a.width <= 2048) {
    start(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  } else {
    start(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  }
  return hipGetLastError();
}

hipError_t launch_combine_backward(const RouteArgs& all, hipStream_t s) {
  return in_parts(all, [&](const RouteArgs& a) { return launch_combine_backward_part(a, s); });
}

}  // namespace she
