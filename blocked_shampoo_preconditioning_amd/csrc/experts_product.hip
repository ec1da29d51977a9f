// The 8-bit products on the matrix cores: y and dx by rows of tokens against one
// matrix an expert, dW over an expert's rows.
//
// Both operands lie along K, 128 values with one scale, which is what one
// instruction of 16 x 16 x 128 takes: it multiplies by the two scales itself, so
// the sums stay in its accumulators from the first K block to the last and no
// other instruction touches them. bf16 results come from there. Inside, it adds
// the products of eight k with what lies 14 bits and more below the largest of
// them cut off, and the groups' sums in fp32 (measured on single products; 1.5e-5
// of the terms' root sum of squares for terms of one size, whatever K). That is a
// hundredth of what rounding to bf16 leaves, and where one term stands out, less
// than a seventieth of what its own rounding to 8 bits does. It is too much for
// fp32 results: those come from the bf16 instruction with both operands widened,
// scales included, which is exact, at a quarter of the rate. There 64 instructions of
// a step come with 128 that widen, two behind each; bytes are read a phase before
// (1536 x 4096 x 2688: 38 us; with four steps in LDS 41, and 47 with bytes widened as
// they are read).
//
// What bounds it: large bf16 products the power limit, near the rate of the library's
// 8-bit product without blocks' scales (in turn on one card, median launch: y of 8192 x
// 2048 x 8192 132 us, 2.1 PFLOP/s, the library 125; of 4096 x 8192 x 2048 67, the library
// 72). Under that limit launches of the former go from 116 us to 152; within a training step
// it takes 123, and its dx and dW 213 (2.6 PFLOP/s). Where each CU has one 128 tile, the
// L2s: 33 KB a step and CU in 0.53 us are 15 TB/s. fp32: the issue of one wave's
// instructions, a step of one tile 1.0 us alone on a CU, 0.75 with two, 0.45 were it the
// matrix cores.
//
// Operands go from HBM to LDS by direct loads of 16 bytes a lane, a K block a step;
// the scales of a step go the same way, 256 bytes an operand. A step's products are
// four phases (halves of A by halves of B), and each phase's fragments are read
// while the one before multiplies, also across the barrier, which sits in the
// middle: before it the step's last reads are done and the next step has landed,
// after it the step's place is loaded again.
//
// A workgroup stays on its CU and goes through tile after tile, of one product or
// two, by records that the launch before has written. To the loads a tile's last
// step is followed by the next tile's first, so that results are stored while the
// next operands are on their way.
#include <type_traits>
#include <utility>

#include "experts_device.h"

namespace she {

using shl::floatx4;
using shl::store8;

namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) const int4v* lds_int4;
typedef __attribute__((address_space(3))) const uint32_t* lds_word;

template <int N, class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0) .. f(N - 1) with constants: the instruction's scale selectors are part of it.
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of<N>(f, std::make_integer_sequence<int, N>{});
}

// FM x FN operands of 16 rows a wave, WM x WN waves; ST steps' operands in LDS.
template <int FM_, int FN_, int WM_, int WN_, int ST_, bool F32_, int WAVES_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_, NW = WM * WN, NT = 64 * NW;
  static constexpr int ST = ST_;
  static constexpr bool F32 = F32_;
  static constexpr int WAVES = WAVES_;                 // of a SIMD at once
  static constexpr int GROUPS = WAVES * 4 / NW;        // workgroups of a CU at once
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int A_SCALES = A_BYTES + B_BYTES, B_SCALES = A_SCALES + 256;
  static constexpr int STAGE = B_SCALES + 256;
  static_assert(BM <= 256 && BN <= 256 && NW >= 2, "");
};

// A buffer of `size` bytes from base; loads past it give zeros.
__device__ __forceinline__ int4v make_rsrc(uint64_t base, uint32_t size) {
  int4v r;
  r[0] = static_cast<int>(base);
  r[1] = static_cast<int>(base >> 32);
  r[2] = static_cast<int>(size);
  r[3] = 0x00020000;
  return r;
}

// 64 x 16 or 4 bytes from rsrc + soff + voff (a lane's own) to LDS at `lds` + plus + 16 or
// 4 * lane; waited for at the next step's barrier. As asm because the compiler
// would wait for every such load before any LDS read; it has no register results.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const int4v& rsrc, uint32_t voff, uint32_t soff, uint32_t lds, int plus) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff), "i"(plus)
               : "memory", "scc", "m0");
}
__device__ __forceinline__ void load_lds4(const int4v& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// An operand of 16 rows: 32 of a row's 128 values a lane.
template <bool F32>
struct Fragment {
  int4v lo, hi;
};
template <>
struct Fragment<true> {
  bf16x8 k[4];
};

// What this launch does not write, read by the scalar unit: a vector load would wait
// for all operands that are on their way.
typedef __attribute__((ext_vector_type(16))) int int16v;
template <class V>
__device__ __forceinline__ V scalar_load(const void* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) V*>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ uint64_t address(int low, int high) { return static_cast<uint64_t>(static_cast<uint32_t>(high)) << 32 | static_cast<uint32_t>(low); }

// Where a wave turns its fp32 results: eight rows of 64.
constexpr int kTurnedPitch = 272, kTurned = 8 * kTurnedPitch;

// Four fp32 of a row, or its last n < 4.
__device__ __forceinline__ void store4(char* p, int64_t off, int n, const floatx4& v) {
  float* q = reinterpret_cast<float*>(p) + off;
  if (n == 4) {
    __builtin_memcpy(q, &v, 16);
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) q[k] = v[k];
}

template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void product_kernel(Products all) {
  constexpr bool F32 = T::F32;
  __shared__ __attribute__((aligned(1024))) char lds[T::ST * T::STAGE];
  __shared__ __attribute__((aligned(16))) char turned[F32 ? T::NW * kTurned : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;
  // Workgroups go round the 8 XCDs, and through the list of their XCD's tiles to and
  // fro: one that has the first of a round has the last of the next.
  const WorkRecord* mine = all.work + static_cast<int64_t>(blockIdx.x % 8) * all.per;
  auto place = [&](int round) {
    const int stride = static_cast<int>(gridDim.x / 8), nth = static_cast<int>(blockIdx.x / 8);
    return round & 1 ? (round + 1) * stride - 1 - nth : round * stride + nth;
  };

  // A load instruction covers eight rows of 128 bytes: row (instruction * NW + wave)
  // * 8 + lane / 8, place lane % 8. A row's chunk c of 16 bytes sits at place c ^
  // swizzle, so that the rows that one read takes together (row r of an operand,
  // which operand_row sends to row (r & 3) + 16 (r >> 2) + ..) fall on different
  // banks: 6.1 cycles a read where (r & 7) ^ (r >> 3) takes 8.4 and none 16.3.
  auto swizzle = [](int r16) { return r16 & 6; };
  constexpr int NA = T::BM / 8 / T::NW, NB = T::BN / 8 / T::NW;
  uint32_t va[NA], vb[NB];
  auto row_off = [&](int j, int64_t pitch) {
    const int row = (j * T::NW + wave) * 8 + (lane >> 3);
    const int r16 = (row & 3) | ((row >> 4) & 3) << 2;
    return static_cast<uint32_t>(row * static_cast<uint32_t>(pitch) + (((lane & 7) ^ swizzle(r16)) << 4));
  };
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char*)lds));

  // Where the loads are: a tile, its buffers, which begin at its first row and K
  // block, and a step of it, which goes into the loads' scalar offset: every
  // instruction here is paid for in every K step. Scales: a wave takes A's (even) or
  // B's, by 4 bytes a lane; those of weights, one for 128 x 128, come as words of four
  // K blocks, from which `pick` takes the step's for all four of a word's places.
  const bool b_scales = wave & 1;
  int4v ra = make_rsrc(0, 0), rb = ra, rs = ra;
  uint32_t vs = 0, scale_step = 0;
  int lround = 0, lproduct = -1, lstep = 0, lturns = 0;
  bool lwords = false, lwords_mine = false;
  auto enter = [&]() __attribute__((always_inline)) {  // the next tile that has steps
    int16v w = {};
    int turns = kNoTileNorBehind;
    do {
      const int at = place(lround++);
      if (at < all.per) w = scalar_load<int16v>(mine + at);
      turns = at < all.per ? w[14] : kNoTileNorBehind;
    } while (turns == 0 || turns == kNoTile);
    const bool more = turns > 0;
    const int product = more ? w[15] >> 22 : 0;
    const ProductArgs& g = all.p[product];
    if (product != lproduct) {
#pragma unroll
      for (int j = 0; j < NA; ++j) va[j] = row_off(j, g.pitch);
#pragma unroll
      for (int j = 0; j < NB; ++j) vb[j] = row_off(j, g.pitch);
      lproduct = product;
    }
    // where nothing is left the loads give zeros
    ra = make_rsrc(address(w[0], w[1]), more ? w[4] : 0);
    rb = make_rsrc(address(w[2], w[3]), more ? w[5] : 0);
    rs = make_rsrc(b_scales ? address(w[8], w[9]) : address(w[6], w[7]), !more ? 0 : b_scales ? w[11] : w[10]);
    lwords = w[15] >> 20 & 1;
    lwords_mine = lwords && b_scales;
    // words: each half of a wave those of its 128 columns
    vs = lwords_mine ? lane >> 5 && w[15] >> 21 & 1 ? static_cast<uint32_t>(g.b_scale_pitch) : 0u : lane * 4;
    scale_step = static_cast<uint32_t>(b_scales ? g.b_blocks : g.a_blocks) * kBlock;
    lturns = more ? turns : 0x7fffffff;
    lstep = 0;
  };
  uint32_t at = 0, ks = 0, ss = 0;
  uint32_t picks[T::ST + 1];  // of the steps from the one that is read on
  auto aim = [&](int buf) {
    at = lds_base + buf * T::STAGE;
    ks = static_cast<uint32_t>(lstep) * kBlock;
    ss = lwords_mine ? static_cast<uint32_t>(lstep) & ~3u : static_cast<uint32_t>(lstep) * scale_step;
    picks[T::ST] = lwords ? static_cast<uint32_t>(lstep & 3) * 0x01010101u : 0x03020100u;
    ++lstep;
  };
  auto load = [&](int q) {
    if (q < NA)
      load_lds16(ra, va[q], ks, at + wave * 1024, q * T::NW * 1024);
    else if (q < NA + NB)
      load_lds16(rb, vb[q - NA], ks, at + wave * 1024, T::A_BYTES + (q - NA) * T::NW * 1024);
    else
      load_lds4(rs, vs, ss, at + (b_scales ? T::B_SCALES : T::A_SCALES));
  };
  constexpr int kLoads = NA + NB + 1;
  auto next_pick = [&]() {
#pragma unroll
    for (int i = 0; i < T::ST; ++i) picks[i] = picks[i + 1];
  };

  // A lane's places in the reads: row r16 of an operand, chunks q4 and q4 + 4.
  const int r16 = lane & 15, q4 = lane >> 4;
  const uint32_t chunk = (q4 ^ swizzle(r16)) << 4;
  const int lane_row = 16 * (r16 >> 2) + (r16 & 3);
  uint32_t fa = lds_base + (wm * T::FM * 16 + lane_row) * 128 + chunk;
  uint32_t fb = lds_base + T::A_BYTES + (wn * T::FN * 16 + lane_row) * 128 + chunk;
  uint32_t fsa = lds_base + T::A_SCALES + (wm * T::FM * 16 & ~127) + r16 * 8 + (T::FM == 4 ? (wm & 1) * 4 : 0);
  uint32_t fsb = lds_base + T::B_SCALES + (wn * T::FN * 16 & ~127) + r16 * 8 + (T::FN == 4 ? (wn & 1) * 4 : 0);
  int rbuf = 0;  // the buffer that is read
  auto other_buffer = [&]() {
    const uint32_t by = ++rbuf == T::ST ? 0u - (T::ST - 1) * T::STAGE : static_cast<uint32_t>(T::STAGE);
    if (rbuf == T::ST) rbuf = 0;
    fa += by, fb += by, fsa += by, fsb += by;
  };

  // scales: operand f's in byte f % 4 of word f / 4; those of the step that is
  // multiplied, and those of the step that is read
  constexpr int SA = T::FM / 4, SB = T::FN / 4;
  uint32_t sa[SA], sb[SB], sa2[SA], sb2[SB];
  auto read_scales = [&]() {
#pragma unroll
    for (int i = 0; i < SA; ++i) sa2[i] = *reinterpret_cast<lds_word>(fsa + 4 * i);
#pragma unroll
    for (int i = 0; i < SB; ++i) sb2[i] = *reinterpret_cast<lds_word>(fsb + 4 * i);
  };
  auto use_scales = [&]() {
#pragma unroll
    for (int i = 0; i < SA; ++i) sa[i] = sa2[i];
#pragma unroll
    for (int i = 0; i < SB; ++i) sb[i] = __builtin_amdgcn_perm(sb2[i], sb2[i], picks[0]);
  };
  auto scale_a = [&](int i) { return value_of(sa2[i >> 2] >> (8 * (i & 3)) & 255u); };
  auto scale_b = [&](int j) { return value_of(__builtin_amdgcn_perm(sb2[j >> 2], sb2[j >> 2], picks[0]) >> (8 * (j & 3)) & 255u); };
  // half of operand f: chunk q4 or q4 + 4 of its row
  auto fetch = [&](uint32_t base, int f, int half) {
    const uint32_t from = base + (64 * (f >> 2) + 4 * (f & 3)) * 128;
    return *reinterpret_cast<lds_int4>(half ? from ^ 64u : from);
  };

  floatx4 acc[T::FM][T::FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  };

  constexpr int HA = T::FM / 2, HB = T::FN / 2, kMma = HA * HB;
  Fragment<F32> a0[HA], a1[HA], b0[HB], b1[HB];
  // One phase: products of half IH of A and half JH of B, with more(q) behind the q-th
  // instruction. fp32: four an operand pair, those of one pair not behind each other.
  constexpr int kSlots = F32 ? 4 * kMma : kMma;
  auto phase = [&](auto ih, auto jh, const Fragment<F32>(&x)[HA], const Fragment<F32>(&y)[HB], auto&& more) {
    each<kSlots>([&](auto q) {
      constexpr int Q = decltype(q)::value, i = Q % kMma / HB, j = Q % HB, I = decltype(ih)::value * HA + i, J = decltype(jh)::value * HB + j;
      if constexpr (F32) {
        acc[I][J] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[j].k[Q / kMma], x[i].k[Q / kMma], acc[I][J], 0, 0, 0);
      } else {
        const int8v av = __builtin_shufflevector(x[i].lo, x[i].hi, 0, 1, 2, 3, 4, 5, 6, 7);
        const int8v bv = __builtin_shufflevector(y[j].lo, y[j].hi, 0, 1, 2, 3, 4, 5, 6, 7);
        acc[I][J] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc[I][J], 0, 0, J & 3, static_cast<int>(sb[J >> 2]), I & 3,
                                                                     static_cast<int>(sa[I >> 2]));
      }
      more(Q);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // A phase's reads of a half of A or B, spread over the first three quarters of
  // its products: four waves that read two at a time would wait for the LDS.
  auto reads = [&](auto count, int q, auto&& read) {
    constexpr int N = 2 * decltype(count)::value, SPAN = kMma * 3 / 4 > 0 ? kMma * 3 / 4 : 1;
#pragma unroll
    for (int r = 0; r < N; ++r)
      if (r * SPAN / N == q) read(r >> 1, r & 1);
  };
  auto read_a = [&](Fragment<F32>(&x)[HA], int first, int q) {
    if constexpr (!F32) reads(std::integral_constant<int, HA>{}, q, [&](int i, int half) { (half ? x[i].hi : x[i].lo) = fetch(fa, first + i, half); });
  };
  auto read_b = [&](Fragment<F32>(&x)[HB], int first, int q) {
    if constexpr (!F32) reads(std::integral_constant<int, HB>{}, q, [&](int j, int half) { (half ? x[j].hi : x[j].lo) = fetch(fb, first + j, half); });
  };
  // fp32: bytes are read a phase before they are widened, four reads a half of an
  // operand, and widened a word (of 4 HA) at a time, as many as go behind an instruction.
  static_assert(!F32 || HA == HB, "");
  constexpr int kHeld = F32 ? 2 * HA : 1, kWords = 4 * kHeld;
  int4v held[2][kHeld];
  auto hold_a = [&](int4v(&v)[kHeld], int first, int r) {
    if (r >= 0 && r < kHeld) v[r] = fetch(fa, first + r / 2, r & 1);
  };
  auto hold_b = [&](int4v(&v)[kHeld], int first, int r) {
    if (r >= 0 && r < kHeld) v[r] = fetch(fb, first + r / 2, r & 1);
  };
  auto widen_word = [&](Fragment<F32>& x, const int4v& v, int half, int w, float scale) {
    if constexpr (F32) widen(v[w], scale, x.k[2 * half + w / 2], 4 * (w & 1));
  };
  auto widen_a = [&](Fragment<F32>(&x)[HA], const int4v(&v)[kHeld], int first, int w) {
    if (w >= 0 && w < kWords) widen_word(x[w / 8], v[w / 4], w / 4 & 1, w & 3, scale_a(first + w / 8));
  };
  auto widen_b = [&](Fragment<F32>(&x)[HB], const int4v(&v)[kHeld], int first, int w) {
    if (w >= 0 && w < kWords) widen_word(x[w / 8], v[w / 4], w / 4 & 1, w & 3, scale_b(first + w / 8));
  };
  const std::integral_constant<int, 0> first{};
  const std::integral_constant<int, 1> second{};

  // the tile that is multiplied: c, turns and shape of its record
  int round = 0, turns = kNoTileNorBehind, turn = 0;
  int4v c{};
  auto next_tile = [&]() __attribute__((always_inline)) {
    do {
      const int at = place(round++);
      if (at < all.per) c = scalar_load<int4v>(&mine[at].c);
      turns = at < all.per ? c[2] : kNoTileNorBehind;
    } while (turns == kNoTile);
    turn = 0;
  };
  next_tile();
  if (turns == kNoTileNorBehind) return;

  // the first tiles' first steps; their first fragments
#pragma unroll 1
  for (int i = 0; i < T::ST; ++i) {
    if (lstep == lturns) enter();
    aim(i);
    next_pick();
#pragma unroll
    for (int q = 0; q < kLoads; ++q) load(q);
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((T::ST - 1) * kLoads) : "memory");
  read_scales();
  if constexpr (F32) {
#pragma unroll
    for (int r = 0; r < kHeld; ++r) hold_a(held[0], 0, r), hold_b(held[1], 0, r);
#pragma unroll
    for (int w = 0; w < kWords; ++w) widen_a(a0, held[0], 0, w), widen_b(b0, held[1], 0, w);
#pragma unroll
    for (int r = 0; r < kHeld; ++r) hold_b(held[0], HB, r);
  } else {
#pragma unroll
    for (int q = 0; q < kMma; ++q) {
      read_a(a0, 0, q);
      read_b(b0, 0, q);
    }
    use_scales();
  }
  __builtin_amdgcn_sched_barrier(0);
  int buf = 0;
  bool stores = false;  // whether some may be behind the loads that are out
#pragma unroll 1
  do {
    clear();
    // as many steps as neither the loads nor the products leave their tile
#pragma unroll 1
    while (turn < turns) {
      if (lstep == lturns) enter();
      const int until = turn + min(turns - turn, lturns - lstep);
#pragma unroll 1
      for (; turn < until; ++turn) {
        phase(first, first, a0, b0, [&](int q) {
          if (q == 0) aim(buf);
          if constexpr (F32) {
            hold_a(held[1], HA, q);
            widen_b(b1, held[0], HB, q);
          } else {
            read_b(b1, HB, q);
          }
        });
        phase(first, second, a0, b1, [&](int q) {
          if constexpr (F32)
            widen_a(a1, held[1], HA, q);
          else
            read_a(a1, HA, q);
        });
        other_buffer();
        // the next step has landed: what is still out are the loads of those behind it
        if (T::ST > 2 && !stores)
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((T::ST - 2) * kLoads) : "memory");
        else
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        stores = false;
        // the next step's first fragments, and the loads of the one that takes this one's place
        auto loads_at = [&](int q) {
#pragma unroll
          for (int e = 0; e < kLoads; ++e)
            if (e * 2 * kSlots / kLoads == q) load(e);
        };
        if (++buf == T::ST) buf = 0;
        next_pick();
        phase(second, first, a1, b0, [&](int q) {
          if (q == 0) read_scales();
          if constexpr (F32) {
            hold_a(held[0], 0, q);
            hold_b(held[1], 0, q - kHeld);
            const int w = 2 * (q - kSlots / 2);
            widen_a(a0, held[0], 0, w), widen_a(a0, held[0], 0, w < 0 ? -1 : w + 1);
          } else {
            read_a(a0, 0, q);
          }
          loads_at(q);
        });
        phase(second, second, a1, b1, [&](int q) {
          if constexpr (F32) {
            hold_b(held[0], HB, q);
            widen_b(b0, held[1], 0, q);
          } else {
            read_b(b0, 0, q);
          }
          loads_at(kSlots + q);
        });
        if constexpr (!F32) use_scales();
      }
    }

    // A lane's accumulators of four operands of B are 16 consecutive columns of a row.
    char* out = reinterpret_cast<char*>(address(c[0], c[1]));
    const int rows = c[3] & 1023, cols = c[3] >> 10 & 1023;
    const int64_t ldc = all.p[c[3] >> 22].ldc;
    if constexpr (F32) {
      // By way of LDS, so that 16 lanes write a row's 256 bytes at once: four pieces of
      // 16 bytes out of every 64, as they lie in the accumulators, are four requests
      // to the L2 (3000 x 128 x 2688: 12.4 us, without 17.5). 32 bytes of bf16 are not
      // worth the way.
      int from = lane >> 4, col0 = wn * T::FN * 16 + (lane & 15) * 4;
      asm volatile("" : "+v"(from), "+v"(col0));
      char* mine = turned + wave * kTurned;
#pragma unroll
      for (int i = 0; i < T::FM; ++i) {
        const int row0 = wm * T::FM * 16 + 64 * (i >> 2) + 4 * (i & 3);
        if (row0 >= rows) continue;
#pragma unroll
        for (int J = 0; J < T::FN / 4; ++J) {
          const int col = col0 + 64 * J, n = min(4, cols - col);
#pragma unroll
          for (int part = 0; part < 2; ++part) {  // eight of the operand's rows
            if (r16 >> 3 == part) {
#pragma unroll
              for (int h = 0; h < 4; ++h) *reinterpret_cast<floatx4*>(mine + (r16 & 7) * kTurnedPitch + q4 * 64 + 16 * h) = acc[i][4 * J + h];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = 8 * part + 4 * k + from, row = row0 + 16 * (r >> 2) + (r & 3);
              const floatx4 v = *reinterpret_cast<const floatx4*>(mine + (4 * k + from) * kTurnedPitch + (lane & 15) * 16);
              if (row < rows && n > 0) store4(out, row * ldc + col, n, v);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
          }
        }
      }
    } else {
      // (not to be worked out ahead of the loop: registers are for its operands)
      int row0 = wm * T::FM * 16 + lane_row, col0 = wn * T::FN * 16 + 16 * q4;
      asm volatile("" : "+v"(row0), "+v"(col0));
#pragma unroll
      for (int i = 0; i < T::FM; ++i) {
        const int row = row0 + 64 * (i >> 2) + 4 * (i & 3);
        if (row >= rows) continue;
#pragma unroll
        for (int J = 0; J < T::FN / 4; ++J) {
          const int col = col0 + 64 * J;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = acc[i][4 * J + 2 * h + q / 4][q % 4];
            const int n = min(8, cols - col - 8 * h);
            if (n > 0) store8(out, row * ldc + col + 8 * h, n, false, v);
          }
        }
      }
    }
    stores = true;
    next_tile();
  } while (turns != kNoTileNorBehind);
  // the last loads (zeros) have landed
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <class T>
void start(const Products& a, hipStream_t s) {
  // as many workgroups as the card takes at once
  const int fit = 32 * T::GROUPS;
  const uint32_t grid = static_cast<uint32_t>(8 * (a.per < fit ? a.per : fit));
  if (grid) product_kernel<T><<<grid, T::NT, 0, s>>>(a);
}

}  // namespace

hipError_t launch_products(const Products& a, hipStream_t s) {
  if (a.f32)
    start<Tile<4, 4, 2, 2, 2, true, 2>>(a, s);
  else if (a.tile == kProduct256)
    start<Tile<8, 8, 2, 2, 2, false, 1>>(a, s);
  else if (a.tile == kProduct128Deep)
    start<Tile<4, 4, 2, 2, 4, false, 1>>(a, s);
  else
    start<Tile<4, 4, 2, 2, 2, false, 2>>(a, s);
  return hipGetLastError();
}

}  // namespace she
