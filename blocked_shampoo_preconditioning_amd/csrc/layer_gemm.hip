// The gated feed-forward block's products on the 16-bit matrix cores.
//
// One tiled product serves the block's six: forward [g u] = x [Wg Wu] and
// y = h Wd; backward dh = dy Wd^T, dx = dg Wg^T + du Wu^T, [dWg dWu] = x^T [dg
// du] and dWd = h^T dy. Operands go from HBM to LDS without passing
// registers (buffer loads with an LDS destination, 16 bytes a lane), double
// buffered over K steps of 64; fragments leave LDS as 16-byte rows (K
// contiguous) or through the transposing 8-byte read (K the slow index), so no
// operand is ever transposed in memory. fp32 operands come as three bf16 planes
// whose sum is the value exactly (split3), at every exponent: no element's digits
// go by what the others hold, as one scale for an array would have it. A product
// of two is six products of planes (the three left out are below 2^-25 of it
// together); all six take their fragments from one K step's planes in
// LDS, so a result costs six times the matrix instructions of bf16, but three
// times the loads.
//
// What bounds it: large products run into the power limit (8192 x 2048 x 8192
// bf16, all six: 2.09 ms, 1180 TFLOP/s; the clock falls to 1.9 GHz and the matrix
// cores are busy 62% of the time in the last three products, 38% in dh with its
// epilogue; other schedules of the loop change nothing there), ordinary ones the
// L2s, which feed a 128 tile 32 KiB a K step (0.46 us with every CU busy, 14 TB/s,
// half the rate of the matrix cores), small ones what a launch costs besides its
// K loop: about 9 us from the first load to the last store. Step of 4096 x 768 x
// 2048 bf16 156 us (743 TFLOP/s), 1024 x 768 x 2048 75 us. fp32 4096 x 768 x 2048
// 620 us (187 TFLOP/s of fp32 results; the library's fp32 product alone: 154), 2048
// x 2048 x 8192 3.0 ms (205; 1230 of bf16 products, the power limit). Two fp16
// planes under one power of two for an operand took 480 us, but rows 10^9 times
// smaller than the largest kept three digits and at 10^12 none.
#include <type_traits>

#include "layer_epilogue.h"
#include "layer_kernels.h"

namespace shl {

namespace {

typedef __attribute__((ext_vector_type(4))) int int4v;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short short4v;
typedef __attribute__((address_space(3))) char lds_char;

constexpr uint32_t kOutOfRange = 0x80000000u;

// ------------------------------------------------------------------ the tile
// WM x WN waves of FM x FN fragments of 16 x 16. With KG = 2 there are two such
// sets of waves, each with half of the K steps and buffers of its own, whose
// sums are joined through LDS: four waves alone on a CU leave its matrix cores
// idle between their phases (a 128 tile takes 0.6 us a K step with them, half of
// 0.85 with eight; y of 4096 x 2048 x 768, 192 tiles: 26.5 against 22.8 us).
// P planes of an operand (planes(f32)); the K step BK is 32 for three, so that
// two steps of 128 x 256 results fit in LDS.
constexpr int k_step(bool f32) { return f32 ? 32 : 64; }
template <int FM_, int FN_, int WM_, int WN_, int KG_, bool F32_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_, KG = KG_;
  static constexpr bool F32 = F32_;
  static constexpr int P = planes(F32), BK = k_step(F32);
  static constexpr int NW = WM * WN, NT = NW * 64 * KG;
  static_assert(KG == 1 || (KG == 2 && FM == 4 && !F32), "");
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;  // one plane's
  static constexpr int STAGE = P * (A_BYTES + B_BYTES);
  static constexpr int PITCH = FN * 16 + 4;  // floats of a row of the epilogue's strips
  static constexpr int STRIPS = NT / 64 * 32 * PITCH * 4;
  static constexpr int LDS = KG * 2 * STAGE > STRIPS ? KG * 2 * STAGE : STRIPS;
  static constexpr int WAVES = 160 * 1024 / LDS * NT / 256;  // of a SIMD at once
};

// LDS order of 16-byte chunks. A row operand's tile is [rows][BK k] (8 or 4
// chunks a row), a column operand's [BK k][width] (16 or 8 chunks a row). Chunk c
// of row r sits at place c ^ swizzle(r), so that the rows that one read takes
// together fall on different banks, whether the LDS serves 128 or 256 bytes
// at a time.
template <int BK>
__device__ __forceinline__ int swz_row(int r) {
  return BK == 64 ? (r & 7) ^ ((r >> 3) & 1) : ((r >> 1) & 3) ^ ((r >> 3) & 1);
}
template <int WIDTH>
__device__ __forceinline__ int swz_col(int k) {
  return WIDTH == 128 ? ((k & 3) << 1) ^ ((k & 3) << 2) ^ ((k >> 1) & 4) : ((k & 3) << 1) ^ ((k >> 2) & 2);
}

// A buffer of `left` >= 0 bytes from base (2 GiB of them are enough: a tile's
// offsets stay under that); loads past it give zeros. The hardware checks whole
// words, so its length is rounded up to one.
__device__ __forceinline__ int4v make_rsrc(uint64_t base, int64_t left) {
  const uint32_t n = static_cast<uint32_t>(left) + 3u & ~3u;
  int4v r;
  r[0] = static_cast<int>(base);
  r[1] = static_cast<int>(base >> 32);
  r[2] = static_cast<int>(static_cast<uint32_t>(left >> 30) > 1u ? 0x7ffffff0u : n);
  r[3] = 0x00020000;
  return r;
}

// 64 x 16 bytes from rsrc + voff (a lane's own) to LDS at `lds` + plus + 16 *
// lane. Written as asm because the compiler would wait for every such load
// before any transposing LDS read; it has no register results, and its arrival
// is waited for at the barrier of the next K step.
// The compiler allots m0 itself and warns of any mention of it; what it knows of
// its changes it needs all the same.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(const int4v& rsrc, uint32_t voff, uint32_t lds, int plus) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "i"(plus)
               : "memory", "scc", "m0");
}
#pragma clang diagnostic pop

typedef __attribute__((address_space(3))) const bf16x8* lds_frag;
typedef __attribute__((address_space(3))) short4v* lds_quad;
__device__ __forceinline__ bf16x8 lds_read16(uint32_t at) { return *reinterpret_cast<lds_frag>(at); }
__device__ __forceinline__ bf16x8 lds_read_tr(uint32_t at, int second) {
  union {
    short4v s[2];
    bf16x8 v;
  } x;
  x.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_quad>(at));
  x.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_quad>(at + second));
  return x.v;
}

// The 16 x 16 x 32 instruction takes less power than the 32 x 32 x 16 one (2090
// against 1860 TFLOP/s sustained from registers), and power is what limits the
// large products.
__device__ __forceinline__ floatx4 mfma(const bf16x8& a, const bf16x8& b, const floatx4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One workgroup's tile (or its part of K) of a product: `block` of `blocks`
// workgroups, a multiple of 8. Forward of 8192 x 2048 x 8192 bf16: g, u and h in
// 522 us (1053 TFLOP/s; 403 MB are written in it), y in 232 (1187); dh with dg and
// du in 340 (808; 268 MB are read and 268 written by its epilogue).
template <class T, bool ACOL, bool BCOL, int EPI>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, uint32_t block, uint32_t blocks, char* lds) {
  constexpr bool GATE = EPI == kGate, F32 = T::F32;
  constexpr int BK = T::BK, P = T::P;
  constexpr int HN = GATE ? T::BN / 2 : T::BN;       // result columns of a tile
  constexpr int BW = GATE ? T::BN / 2 : 128;         // width of a B panel
  static_assert(BW == 128 || BW == 64, "");
  static_assert(!GATE || BCOL, "");
  const int lane = threadIdx.x & 63;
  const int any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kgroup = any_wave / T::NW, wave = any_wave - kgroup * T::NW;
  const int wm = wave % T::WM, wn = wave / T::WM;

  // Workgroups go round the 8 XCDs; each XCD takes a contiguous range of the
  // work, in groups of four row tiles, so that the tiles in flight on one XCD
  // share their operands in its L2.
  const int tm = (g.M + T::BM - 1) / T::BM, tn = (g.N + HN - 1) / HN;
  const uint32_t per = blocks / 8;
  uint32_t id = block % 8 * per + block / 8;
  const uint32_t tiles = static_cast<uint32_t>(tm) * tn;
  if (id >= tiles * g.problems * g.splits) return;
  int split = 0, problem = 0;
  if (g.splits > 1) {
    split = id / (tiles * g.problems);
    id -= split * (tiles * g.problems);
  }
  if (g.problems > 1 && id >= tiles) {
    problem = 1;
    id -= tiles;
  }
  const uint32_t group = id / (4 * static_cast<uint32_t>(tn));
  const uint32_t in_group = min(4u, tm - 4 * group);
  id -= group * 4 * tn;
  const uint32_t tcol = id / in_group;
  const int m0 = (4 * group + id - tcol * in_group) * T::BM, n0 = tcol * HN;

  // K steps of this split, cut as evenly as they go
  const int ksteps = (g.K + BK - 1) / BK, steps = ksteps * g.nseg;
  int first = 0, last = steps;
  if (g.splits > 1) {
    const int each = steps / g.splits, rest = steps - each * g.splits;
    first = each * split + min(split, rest);
    last = first + each + (split < rest ? 1 : 0);
  }
  // the second set of waves may have a step less: it adds zeros in its last one
  const int turns = (last - first + T::KG - 1) / T::KG;
  first += kgroup * turns;
  int loads = min(turns, last - first);  // steps still to be loaded

  // Loads: 1 KiB an instruction, NW instructions at a time, plane after plane. A
  // row operand's buffer starts at the tile's first row and its offsets move along
  // K; a column operand's starts at the step's first K row and its offsets stay.
  constexpr int NAP = T::A_BYTES / 1024 / T::NW, NBP = T::B_BYTES / 1024 / T::NW;  // of one plane
  constexpr int NA = P * NAP, NB = P * NBP;
  constexpr int APP = 128 * BK * 2 / 1024 / T::NW, BPP = BW * BK * 2 / 1024 / T::NW;  // of one panel
  static_assert(APP > 0 && BPP > 0 && NAP > 0, "");
  constexpr int CPR = BK / 8, RPI = 64 / CPR;  // row operand: chunks a row, rows an instruction
  const int64_t lda2 = g.lda * 2, ldb2 = g.ldb * 2;
  // row operand: row (instruction * NW + wave) * RPI + lane / CPR, chunk lane % CPR (swizzled)
  const int rchunk = (lane % CPR) ^ swz_row<BK>(lane / CPR + RPI * wave);
  auto row_off = [&](int64_t ld2, int j) {
    return static_cast<uint32_t>(((j * T::NW + wave) * RPI + lane / CPR) * ld2 + rchunk * 16);
  };
  // column operand of panels `width` wide: K row of the panel, chunk (swizzled)
  auto col_off = [&](int64_t ld2, int width, int j, int panel) {
    const int per_row = width / 8, rows = 64 / per_row;
    const int k = (j * T::NW + wave) * rows + lane / per_row;
    const int c = (lane % per_row) ^ (width == 128 ? swz_col<128>(k) : swz_col<64>(k));
    return static_cast<uint32_t>(k * ld2 + c * 16 + panel * width * 2);
  };
  uint32_t va[NAP], vb[NBP];
#pragma unroll
  for (int j = 0; j < NAP; ++j) va[j] = ACOL ? col_off(lda2, 128, j % APP, j / APP) : row_off(lda2, j);
#pragma unroll
  for (int j = 0; j < NBP; ++j) vb[j] = BCOL ? col_off(ldb2, BW, j % BPP, GATE ? 0 : j / BPP) : row_off(ldb2, j);
  const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char*)lds)) + kgroup * (2 * T::STAGE);
  const uint32_t lds0 = lds_base + wave * 1024;
  const int64_t a_start = ACOL ? 2 * static_cast<int64_t>(m0) : m0 * lda2;
  const int64_t b_start = BCOL ? 2 * static_cast<int64_t>(n0) : n0 * ldb2;
  const int64_t a_size = (ACOL ? (static_cast<int64_t>(g.k_real) - 1) * lda2 + 2 * static_cast<int64_t>(g.M)
                               : (static_cast<int64_t>(g.M) - 1) * lda2 + 2 * static_cast<int64_t>(g.K)) - a_start;
  const int64_t b_size = (BCOL ? (static_cast<int64_t>(g.k_real) - 1) * ldb2 + 2 * static_cast<int64_t>(g.N)
                               : (static_cast<int64_t>(g.N) - 1) * ldb2 + 2 * static_cast<int64_t>(g.K)) - b_start;

  // Where the loads are: segment, K of the step, the operands' buffers. Every
  // instruction here is paid for in every K step, so a step moves the buffers by
  // a few scalar additions; a row operand's chunks past K, which only a
  // segment's last step can have, get an offset out of range once.
  const int64_t a_step = ACOL ? BK * lda2 : BK * 2, b_step = BCOL ? BK * ldb2 : BK * 2;
  const int64_t plane_a2 = g.plane_a * 2, plane_b2 = g.plane_b * 2;
  int seg = 0;
  if (first) seg = min(first, steps - 1) / ksteps;
  int k0 = (first - seg * ksteps) * BK;
  uint64_t pa = 0, pb = 0, pb1 = 0;
  int64_t left_a = 0, left_b = 0;
  bool cut = false;
  auto cut_chunks = [&]() {
    const bool now = (!ACOL || !BCOL) && k0 + BK > g.K;
    if (now == cut) return;
    cut = now;
    const uint32_t bit = now && k0 + rchunk * 8 >= g.K ? kOutOfRange : 0u;
#pragma unroll
    for (int j = 0; j < NAP; ++j)
      if (!ACOL) va[j] = (va[j] & ~kOutOfRange) | bit;
#pragma unroll
    for (int j = 0; j < NBP; ++j)
      if (!BCOL) vb[j] = (vb[j] & ~kOutOfRange) | bit;
  };
  auto enter = [&]() {
    const int64_t ka = k0 / BK * a_step, kb = k0 / BK * b_step;
    pa = reinterpret_cast<uint64_t>(g.a[seg]) + a_start + ka;
    pb = reinterpret_cast<uint64_t>(GATE ? g.b[0][seg] : g.b[problem][seg]) + b_start + kb;
    if (GATE) pb1 = reinterpret_cast<uint64_t>(g.b[1][seg]) + b_start + kb;
    left_a = a_size - ka;
    left_b = b_size - kb;
    cut_chunks();
  };
  int4v ra[P], rb[P], rb1[P];
  uint32_t at = 0;
  auto aim = [&](int buf) {
    at = lds0 + buf * T::STAGE;
    // past the last step nothing is read: the buffer gets zeros
#pragma unroll
    for (int p = 0; p < P; ++p) {
      ra[p] = make_rsrc(pa + p * plane_a2, loads > 0 ? left_a : 0);
      rb[p] = make_rsrc(pb + p * plane_b2, loads > 0 ? left_b : 0);
      if (GATE) rb1[p] = make_rsrc(pb1 + p * plane_b2, loads > 0 ? left_b : 0);
    }
  };
  auto load = [&](int q) {
    if (q < NA) {
      const int p = q / NAP, j = q % NAP;
      load_lds(ra[p], va[j], at, p * T::A_BYTES + j * T::NW * 1024);
    } else {
      const int p = (q - NA) / NBP, j = (q - NA) % NBP;
      load_lds(GATE && j >= BPP ? rb1[p] : rb[p], vb[j], at, P * T::A_BYTES + p * T::B_BYTES + j * T::NW * 1024);
    }
  };
  auto advance = [&]() {
    if (--loads <= 0) return;
    k0 += BK;
    if (k0 < g.K) {
      pa += a_step, pb += b_step;
      if (GATE) pb1 += b_step;
      left_a -= a_step, left_b -= b_step;
      if (k0 + BK > g.K) cut_chunks();
    } else {
      ++seg;
      k0 = 0;
      enter();
    }
  };

  // A lane's places in the fragment reads (16 rows or columns x 32 k, eight k of
  // one row a lane), as LDS addresses of the buffer that is read.
  const int r16 = lane & 15, q4 = lane >> 4;
  // row operand: row r16 of a fragment, chunk 4 ks + q4
  auto row_at = [&](uint32_t tile, int row0, int ks) {
    return static_cast<uint32_t>(tile + (row0 + r16) * (2 * BK) + (((4 * ks + q4) ^ swz_row<BK>(r16)) << 4));
  };
  // column operand: k = 32 ks + 8 q4 + (lane % 16) / 4 (+ 4 in the second
  // read), columns 4 (lane % 4) on
  const int kk = 8 * q4 + (r16 >> 2);
  auto col_at = [&](uint32_t tile, int width, int col0) {
    const int c = (col0 >> 3) + ((lane & 3) >> 1);
    const int s = width == 128 ? swz_col<128>(kk) : swz_col<64>(kk);
    return static_cast<uint32_t>(tile + kk * (width * 2) + ((c ^ s) << 4) + (lane & 1) * 8);
  };
  constexpr int KS = BK / 32;
  constexpr uint32_t b_base = P * T::A_BYTES;
  uint32_t fa[ACOL ? T::FM : KS], fb[BCOL ? T::FN : KS];
  if (ACOL) {
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const int row = (wm * T::FM + i) * 16;
      fa[ACOL ? i : 0] = col_at(lds_base + (row >> 7) * (256 * BK), 128, row & 127);
    }
  } else {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) fa[ACOL ? 0 : ks] = row_at(lds_base, wm * T::FM * 16, ks);
  }
  if (BCOL) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
      // kGate: a wave's first half of the fragments gate panel, second: up panel
      constexpr int H2 = T::FN / 2;
      const int col = GATE ? (wn * H2 + j % H2) * 16 : (wn * T::FN + j) * 16;
      const int panel = GATE ? j / H2 : col >> 7;
      fb[BCOL ? j : 0] = col_at(lds_base + b_base + panel * (BW * BK * 2), BW, GATE ? col : col & 127);
    }
  } else {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) fb[BCOL ? 0 : ks] = row_at(lds_base + b_base, wn * T::FN * 16, ks);
  }
  // fragment i of slice ks (32 k) of plane p
  auto frag_a = [&](int i, int ks, int p = 0) {
    if (ACOL) return lds_read_tr(fa[ACOL ? i : 0] + (ks * (32 * 256) + p * T::A_BYTES), 4 * 256);
    return lds_read16(fa[ACOL ? 0 : ks] + (i * (32 * BK) + p * T::A_BYTES));
  };
  auto frag_b = [&](int j, int ks, int p = 0) {
    if (BCOL) return lds_read_tr(fb[BCOL ? j : 0] + (ks * (32 * BW * 2) + p * T::B_BYTES), 4 * BW * 2);
    return lds_read16(fb[BCOL ? 0 : ks] + (j * (32 * BK) + p * T::B_BYTES));
  };
  uint32_t flip = T::STAGE;
  auto other_buffer = [&]() {
#pragma unroll
    for (uint32_t& x : fa) x += flip;
#pragma unroll
    for (uint32_t& x : fb) x += flip;
    flip = 0u - flip;
  };

  floatx4 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // The K loop, software-pipelined. A K step is two slices of 32. In the large
  // tiles a slice is two phases, for want of registers: the fragments of the
  // operand that has more of them come in two halves, the other's whole; in the
  // small ones it is one (H: fragments of the first operand at a time, F: of
  // the other). Each phase's fragments are read from LDS while the matrix cores
  // work on the phase before, also across the barrier between two steps. At the
  // barrier a wave's loads of the next step have landed and its reads of this
  // step are done, so after it the next step can be read and this step's buffer
  // be filled again, which the last phase does with its loads between the
  // products. With three planes a K step is one slice and six phases, the
  // products of two planes; the last of them are the middle planes', whose
  // fragments' registers the next step's first do not need.
  auto prologue = [&](auto first_reads) {
    if (turns > 0) {
      enter();
  #pragma unroll
      for (int i = 0; i < 2; ++i) {
        aim(i);
  #pragma unroll
        for (int q = 0; q < NA + NB; ++q) load(q);
        advance();
      }
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NA + NB) : "memory");
      first_reads();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if constexpr (F32) {
    bf16x8 a[P][T::FM], b[P][T::FN];
    auto read_a = [&](int p) {
#pragma unroll
      for (int i = 0; i < T::FM; ++i) a[p][i] = frag_a(i, 0, p);
    };
    auto read_b = [&](int p) {
#pragma unroll
      for (int j = 0; j < T::FN; ++j) b[p][j] = frag_b(j, 0, p);
    };
    constexpr int kMma = T::FM * T::FN, kReadsA = T::FM * (ACOL ? 2 : 1), kReadsB = T::FN * (BCOL ? 2 : 1);
    auto product = [&](int q, int pa_, int pb_) {
      floatx4& c = acc[q / T::FN][q % T::FN];
      c = mfma(b[pb_][q % T::FN], a[pa_][q / T::FN], c);
    };
    // a phase's products, the LDS reads before them in the program between them
    auto mma = [&](int pa_, int pb_, auto reads) {
      constexpr int kEach = (decltype(reads)::value + kMma / 2 - 1) / (kMma / 2);
#pragma unroll
      for (int q = 0; q < kMma; ++q) product(q, pa_, pb_);
      if constexpr (kEach > 0) {
#pragma unroll
        for (int q = 0; q < kMma; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    prologue([&]() {
      read_a(0);
      read_b(0);
    });
    int buf = 0;
    for (int turn = 0; turn < turns; ++turn) {
      aim(buf);
      buf ^= 1;
      read_b(1);
      read_a(1);
      mma(0, 0, std::integral_constant<int, kReadsA + kReadsB>{});
      read_b(2);
      mma(0, 1, std::integral_constant<int, kReadsB>{});
      read_a(2);
      mma(1, 0, std::integral_constant<int, kReadsA>{});
      mma(0, 2, std::integral_constant<int, 0>{});
      mma(2, 0, std::integral_constant<int, 0>{});
      other_buffer();
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      read_a(0);
      read_b(0);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int kEach = (NA + NB + kMma - 1) / kMma;
#pragma unroll
      for (int q = 0; q < kMma; ++q) {
        product(q, 1, 1);
        if (q * kEach < NA + NB) {
#pragma unroll
          for (int e = 0; e < kEach; ++e)
            if (q * kEach + e < NA + NB) load(q * kEach + e);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      advance();
    }
  } else {
    constexpr bool HALVE_A = T::FM >= T::FN, TWO = T::FM * T::FN > 16;
    constexpr int H = (HALVE_A ? T::FM : T::FN) / (TWO ? 2 : 1), F = HALVE_A ? T::FN : T::FM;
    bf16x8 lo[H], hi[H], full0[F], full1[F];
    auto read_half = [&](int ks, int half, bf16x8(&x)[H]) {
#pragma unroll
      for (int i = 0; i < H; ++i) x[i] = HALVE_A ? frag_a(half * H + i, ks) : frag_b(half * H + i, ks);
    };
    auto read_full = [&](int ks, bf16x8(&x)[F]) {
#pragma unroll
      for (int i = 0; i < F; ++i) x[i] = HALVE_A ? frag_b(i, ks) : frag_a(i, ks);
    };
    constexpr int kMma = H * F;
    auto product = [&](int half, int q, const bf16x8(&x)[H], const bf16x8(&y)[F]) {
      const int h = q / F, f = q % F;
      if (HALVE_A) {
        floatx4& c = acc[half * H + h][f];
        c = mfma(y[f], x[h], c);
      } else {
        floatx4& c = acc[f][half * H + h];
        c = mfma(x[h], y[f], c);
      }
    };
    // one phase's products, with the LDS reads before them in the program spread
    // between them (a read of a row operand is one instruction, of a column
    // operand two)
    constexpr int kHalfReads = H * ((HALVE_A ? ACOL : BCOL) ? 2 : 1), kFullReads = F * ((HALVE_A ? BCOL : ACOL) ? 2 : 1);
    auto mma = [&](int half, const bf16x8(&x)[H], const bf16x8(&y)[F], int reads) {
#pragma unroll
      for (int q = 0; q < kMma; ++q) product(half, q, x, y);
      if (reads == kHalfReads) {
#pragma unroll
        for (int q = 0; q < kMma; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, (kHalfReads + kMma / 2 - 1) / (kMma / 2), 0);
        }
      } else {
#pragma unroll
        for (int q = 0; q < kMma; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, (kHalfReads + kFullReads + kMma / 2 - 1) / (kMma / 2), 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // the same with a step's loads between them
    auto mma_load = [&](int half, const bf16x8(&x)[H], const bf16x8(&y)[F]) {
      constexpr int kEach = (NA + NB + kMma - 1) / kMma;
#pragma unroll
      for (int q = 0; q < kMma; ++q) {
        product(half, q, x, y);
        if (q * kEach < NA + NB) {
#pragma unroll
          for (int e = 0; e < kEach; ++e)
            if (q * kEach + e < NA + NB) load(q * kEach + e);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    prologue([&]() {
      read_half(0, 0, lo);
      read_full(0, full0);
    });
    int buf = 0;
    for (int turn = 0; turn < turns; ++turn) {
      aim(buf);
      buf ^= 1;
      if (TWO) {
        read_half(0, 1, hi);
        mma(0, lo, full0, kHalfReads);
        read_half(1, 0, lo);
        read_full(1, full1);
        mma(1, hi, full0, kHalfReads + kFullReads);
        read_half(1, 1, hi);
        mma(0, lo, full1, kHalfReads);
      } else {
        read_half(1, 0, hi);
        read_full(1, full1);
        mma(0, lo, full0, kHalfReads + kFullReads);
      }
      other_buffer();
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      read_half(0, 0, lo);
      read_full(0, full0);
      __builtin_amdgcn_sched_barrier(0);
      mma_load(TWO ? 1 : 0, hi, full1);
      advance();
    }
  }

  // Epilogue. A lane's accumulators are column r16 (row m of the result) and
  // rows 4 q4 + 0..3 (result columns n) of each fragment: two rows of FN
  // fragments pass through a wave-private LDS strip and come back as eight
  // columns of one row a lane, so that stores are 16 bytes a lane and whole row
  // segments. kActBwd reads g and u one strip ahead, since a load waits for the
  // stores before it (fp32: its own strip, for want of registers).
  constexpr int AHEAD = F32 ? 0 : 1;
  constexpr int PITCH = T::PITCH;
  constexpr int COLS = GATE ? T::FN * 8 : T::FN * 16;            // result columns of a wave
  constexpr int LR = COLS / 8, RP = 64 / LR, NP = 32 / RP;       // lanes a row, rows a pass, passes
  constexpr int STRIPS = T::FM / 2 / T::KG;                      // of a wave
  const int row0 = m0 + wm * T::FM * 16 + kgroup * 32 + lane / LR;
  const int c8 = (lane % LR) * 8, col = n0 + wn * COLS + c8;
  const int64_t ldc = EPI == kStore && problem ? g.e.ldc1 : g.e.ldc;
  const int64_t oc = row0 * ldc + col, og = row0 * g.e.ldg + col;
  const Activation<F32> act(g.e.act);
  Raw8<F32> gr[1 + AHEAD][NP], ur[1 + AHEAD][NP];
  const bool act_bwd = EPI == kActBwd && g.splits == 1;
  if (act_bwd && AHEAD) {
#pragma unroll
    for (int p = 0; p < NP; ++p) load_gu<F32>(g.e, row0 + p * RP < g.M, og + p * RP * g.e.ldg, col, g.N, gr[0][p], ur[0][p]);
  }
  // the last loads (zeros) have landed and all reads are done: LDS is free
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (T::KG == 2) {
    // each set joins one strip: it gives the other's and takes its own
    floatx4* give = reinterpret_cast<floatx4*>(lds) + any_wave * (2 * T::FN * 64) + lane;
    const floatx4* get = reinterpret_cast<floatx4*>(lds) + (any_wave ^ T::NW) * (2 * T::FN * 64) + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
        give[(h * T::FN + j) * 64] = kgroup ? acc[h][j] : acc[2 + h][j];
        acc[h][j] = kgroup ? acc[2 + h][j] : acc[h][j];
      }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) acc[h][j] += get[(h * T::FN + j) * 64];
    __syncthreads();
  }
  float* strip = reinterpret_cast<float*>(lds) + any_wave * (32 * PITCH);
#pragma unroll
  for (int i = 0; i < STRIPS; ++i) {
    if (act_bwd && i + AHEAD < STRIPS) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        load_gu<F32>(g.e, row0 + (i + AHEAD) * 32 + p * RP < g.M, og + ((i + AHEAD) * 32 + p * RP) * g.e.ldg, col, g.N,
                     gr[(i + AHEAD) & AHEAD][p], ur[(i + AHEAD) & AHEAD][p]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) *reinterpret_cast<floatx4*>(strip + (h * 16 + r16) * PITCH + j * 16 + 4 * q4) = acc[2 * i + h][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    auto strip8 = [&](int p, float(&v)[8], float(&w)[8]) {
      const float* x = strip + (p * RP + lane / LR) * PITCH + c8;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = x[q], w[q] = GATE ? x[COLS + q] : 0.f;
    };
    if (g.splits > 1) {
      constexpr int parts = GATE ? 2 : 1;
      const int64_t plane = static_cast<int64_t>(g.M) * g.N;
      float* part = g.partial + (static_cast<int64_t>(split) * g.problems + problem) * parts * plane + col;
      const int n = min(8, g.N - col);
#pragma unroll 1
      for (int p = 0; p < NP; ++p) {
        const int row = row0 + i * 32 + p * RP;
        float v[8], w[8];
        strip8(p, v, w);
        if (row < g.M && n > 0) {
          store8(part, static_cast<int64_t>(row) * g.N, n, true, v);
          if (GATE) store8(part + plane, static_cast<int64_t>(row) * g.N, n, true, w);
        }
      }
    } else {
      auto pass = [&](int p) {
        const int down = i * 32 + p * RP;
        float v[8], w[8];
        strip8(p, v, w);
        if (row0 + down >= g.M) return;
        finish8<F32, EPI>(g.e, act, problem, oc + down * ldc, og + down * g.e.ldg, col, g.N, v, w, gr[i & AHEAD][p], ur[i & AHEAD][p]);
      };
      if (EPI == kActBwd) {
#pragma unroll
        for (int p = 0; p < NP; ++p) pass(p);
      } else {
#pragma unroll 1
        for (int p = 0; p < NP; ++p) pass(p);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <class T, bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(T::NT, T::WAVES) void gemm_kernel(GemmArgs g) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];
  gemm_tile<T, ACOL, BCOL, EPI>(g, blockIdx.x, gridDim.x, lds);
}

// The backward pass's last three products in one launch: dx (operands by rows),
// dWd, and dWg with dWu (operands by columns). None fills the card alone at
// ordinary sizes (1024..4096 tokens of 768 x 2048: 48..192 tiles of 128), all
// together nearly do, with fewer splits and no gaps between launches (backward
// pass of 1024 tokens 71 -> 47 us, of 4096 142 -> 105). 8192 x 2048 x 8192 bf16:
// 1077 us (1276 TFLOP/s); 4096 x 768 x 2048: 68 us (945).
template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES) void gemm_group_kernel(GroupArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];
  const uint32_t b = blockIdx.x;
  if (b < a.start[1])
    gemm_tile<T, false, false, kStore>(a.g[0], b, a.start[1], lds);
  else if (b < a.start[2])
    gemm_tile<T, true, true, kStore>(a.g[1], b - a.start[1], a.start[2] - a.start[1], lds);
  else
    gemm_tile<T, true, true, kStore>(a.g[2], b - a.start[2], a.start[3] - a.start[2], lds);
}

// Joins the parts of a split product in their order and runs the epilogue. A
// launch and one trip to the caches, which still hold the parts: 1024 x 768 from
// 4 parts 4.1 us, dg and du of 1024 x 2048 fp32 from 2 parts 12.6 us (59 MB).
template <bool F32, int EPI>
__global__ __launch_bounds__(256) void gemm_finish_kernel(GemmArgs g) {
  const int width = max(g.N, g.e.pad_to);
  const int c8 = (width + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int problem = blockIdx.y;
  const int64_t row = i / c8;
  const int col = static_cast<int>(i - row * c8) * 8;
  const int64_t oc = row * (EPI == kStore && problem ? g.e.ldc1 : g.e.ldc) + col, og = row * g.e.ldg + col;
  constexpr int parts = EPI == kGate ? 2 : 1;
  const int64_t plane = static_cast<int64_t>(g.M) * g.N;
  const int n = max(0, min(8, g.N - col));
  if (i < static_cast<int64_t>(c8) * g.M) {
    Raw8<F32> gr, ur;
    if (EPI == kActBwd) load_gu<F32>(g.e, true, og, col, g.N, gr, ur);
    float v[8], w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = w[q] = 0.f;
    const int64_t jump = plane * g.problems * parts;
    const float* p = g.partial + static_cast<int64_t>(problem) * parts * plane;
    constexpr int U = 4;  // parts in flight
    for (int s = 0; s < g.splits; s += U, p += U * jump) {
      Raw8<true> x[U], y[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int m = s + k < g.splits ? n : 0;
        x[k] = fetch8<true>(p + k * jump, row * g.N, col, m);
        if (EPI == kGate) y[k] = fetch8<true>(p + k * jump + plane, row * g.N, col, m);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int m = s + k < g.splits ? n : 0;
        float t[8];
        unpack8<true>(settle8<true>(x[k], col, m), t);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += t[q];
        if (EPI == kGate) {
          unpack8<true>(settle8<true>(y[k], col, m), t);
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] += t[q];
        }
      }
    }
    finish8<F32, EPI>(g.e, Activation<F32>(g.e.act), problem, oc, og, col, g.N, v, w, gr, ur);
  }
}

// ------------------------------------------------------------------- copies
// Row and first column of an operand's i-th group of eight columns, c8 a row. A
// 64-bit division takes longer than the group's load.
__device__ __forceinline__ void group_place(int64_t i, int64_t c8, int64_t total, int64_t& row, int& col) {
  if (total <= 0x7fffffff) {
    const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(c8);
    row = r;
    col = static_cast<int>(static_cast<uint32_t>(i) - r * static_cast<uint32_t>(c8)) * 8;
  } else {
    row = i / c8;
    col = static_cast<int>(i - row * c8) * 8;
  }
}

// Copies operands into rows that loads can take (16-byte aligned, padded with
// zeros to whole 16 bytes); fp32 values become three bf16 planes (split3). Bound
// by HBM: x and the weights of 4096 x 768 x 2048 fp32 (31 MB in, 47 out) in 16.5
// us, bf16 of odd strides (1537 x 1001 x 2730, 39 MB) in 8.
template <bool F32>
__global__ __launch_bounds__(256) void pack_kernel(PackList list) {
  const PackArgs& p = list.t[blockIdx.y];
  const int64_t c8 = p.ld_out / 8, total = c8 * p.rows, plane = p.rows * p.ld_out;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    int64_t row;
    int col;
    group_place(i, c8, total, row, col);
    const int n = static_cast<int>(min<int64_t>(8, p.cols - col));
    const Raw8<F32> raw = load_raw8<F32>(p.src, row * p.ld, col, n);
    if constexpr (F32) {
      float v[8];
      unpack8<F32>(raw, v);
      store_planes(p.out, row * p.ld_out + col, plane, v);
    } else {
      *reinterpret_cast<uint4v*>(p.out + row * p.ld_out + col) = raw.w[0];
    }
  }
}

// 256 tiles run as eight waves of 128 x 64 (kGate: 64 x 128, so that a wave's
// rows of h are whole 128-byte segments). fp32 tiles too run as eight: of 64 x 64
// in the wide one, of 64 x 32 in the other, but for the gate's, whose panels of 64
// columns are loads for four waves (step of 8192 x 256 x 512 with four everywhere
// 223 us, with eight 190; 300 x 512 x 1024 87 and 79).
template <int EPI>
using Tile256 = Tile<EPI == kGate ? 4 : 8, EPI == kGate ? 8 : 4, EPI == kGate ? 4 : 2, EPI == kGate ? 2 : 4, 1, false>;
using Tile128 = Tile<4, 4, 2, 2, 1, false>;
template <int EPI>
using TileF32 = Tile<4, EPI == kGate ? 4 : 2, 2, EPI == kGate ? 2 : 4, 1, true>;
using Tile128x2 = Tile<4, 4, 2, 2, 2, false>;
using TileWide = Tile<4, 4, 2, 4, 1, true>;

// Workgroups of a product, a multiple of 8 (one for each XCD).
int64_t gemm_blocks(const GemmArgs& g, TileKind tile, bool gate) {
  if (g.M <= 0 || g.N <= 0) return 0;
  return (gemm_tiles(g.M, g.N, g.problems, tile, gate) * g.splits + 7) / 8 * 8;
}

template <class T, bool ACOL, bool BCOL, int EPI>
hipError_t launch_one(const GemmArgs& g, TileKind tile, hipStream_t s) {
  const int64_t grid = gemm_blocks(g, tile, EPI == kGate);
  if (grid > 0x7fffffff || gemm_steps(g.K, g.nseg, T::F32) > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_kernel<T, ACOL, BCOL, EPI>), dim3(static_cast<uint32_t>(grid)), dim3(T::NT), 0, s, g);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || g.splits == 1) return err;
  return launch_finish(g, static_cast<Epi>(EPI), s);
}

template <class T>
hipError_t launch_group_tiles(GroupArgs& a, TileKind tile, hipStream_t s) {
  int64_t at = 0;
  for (int i = 0; i < 3; ++i) {
    a.start[i] = static_cast<uint32_t>(at);
    at += gemm_blocks(a.g[i], tile, false);
    if (at > 0x7fffffff || gemm_steps(a.g[i].K, a.g[i].nseg, T::F32) > 0x7fffffff) return hipErrorInvalidValue;
  }
  a.start[3] = static_cast<uint32_t>(at);
  if (at == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_group_kernel<T>), dim3(static_cast<uint32_t>(at)), dim3(T::NT), 0, s, a);
  hipError_t e = hipGetLastError();
  for (int i = 0; i < 3 && e == hipSuccess; ++i)
    if (a.g[i].splits > 1 && a.g[i].M > 0) e = launch_finish(a.g[i], kStore, s);
  return e;
}

template <bool ACOL, bool BCOL, int EPI>
hipError_t launch_tile(const GemmArgs& g, TileKind tile, hipStream_t s) {
  if (g.f32)
    return tile == kTileWide ? launch_one<TileWide, ACOL, BCOL, EPI>(g, tile, s) : launch_one<TileF32<EPI>, ACOL, BCOL, EPI>(g, tile, s);
  return tile == kTile256   ? launch_one<Tile256<EPI>, ACOL, BCOL, EPI>(g, tile, s)
         : tile == kTile128 ? launch_one<Tile128, ACOL, BCOL, EPI>(g, tile, s)
                            : launch_one<Tile128x2, ACOL, BCOL, EPI>(g, tile, s);
}

uint32_t pack_grid(const PackList& l) {
  int64_t most = 1;
  for (int i = 0; i < l.n; ++i) {
    const int64_t b = (l.t[i].rows * (l.t[i].ld_out / 8) + 255) / 256;
    most = b > most ? b : most;
  }
  return static_cast<uint32_t>(most < 4096 ? most : 4096);
}

}  // namespace

int64_t gemm_tiles(int64_t M, int64_t N, int problems, TileKind tile, bool gate) {
  const int64_t h = tile == kTile256 ? 256 : 128, w = tile == kTile256 || tile == kTileWide ? 256 : 128, hn = gate ? w / 2 : w;
  return ((M + h - 1) / h) * ((N + hn - 1) / hn) * problems;
}

int64_t gemm_steps(int64_t K, int nseg, bool f32) { return (K + k_step(f32) - 1) / k_step(f32) * nseg; }

hipError_t launch_gemm(const GemmArgs& g, TileKind tile, bool a_cols, bool b_cols, Epi epi, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
  if (!is_tile(tile, g.f32)) return hipErrorInvalidValue;
  if (!a_cols && b_cols && epi == kGate) return launch_tile<false, true, kGate>(g, tile, s);
  if (!a_cols && b_cols && epi == kStore) return launch_tile<false, true, kStore>(g, tile, s);
  if (!a_cols && !b_cols && epi == kActBwd) return launch_tile<false, false, kActBwd>(g, tile, s);
  return hipErrorInvalidValue;
}

hipError_t launch_group(GroupArgs& a, TileKind tile, bool f32, hipStream_t s) {
  if (!is_tile(tile, f32)) return hipErrorInvalidValue;
  if (f32) return tile == kTileWide ? launch_group_tiles<TileWide>(a, tile, s) : launch_group_tiles<TileF32<kStore>>(a, tile, s);
  return tile == kTile256   ? launch_group_tiles<Tile256<kStore>>(a, tile, s)
         : tile == kTile128 ? launch_group_tiles<Tile128>(a, tile, s)
                            : launch_group_tiles<Tile128x2>(a, tile, s);
}

hipError_t launch_finish(const GemmArgs& g, Epi epi, hipStream_t s) {
  const int64_t c8 = (((g.e.pad_to > g.N) ? g.e.pad_to : g.N) + 7) / 8;
  const dim3 grid(static_cast<uint32_t>((c8 * g.M + 255) / 256), g.problems), block(256);
#define SHL_FINISH(E)                                                                    \
  if (epi == E) {                                                                        \
    if (g.f32)                                                                           \
      hipLaunchKernelGGL((gemm_finish_kernel<true, E>), grid, block, 0, s, g);           \
    else                                                                                 \
      hipLaunchKernelGGL((gemm_finish_kernel<false, E>), grid, block, 0, s, g);          \
    return hipGetLastError();                                                            \
  }
  SHL_FINISH(kStore)
  SHL_FINISH(kGate)
  SHL_FINISH(kActBwd)
#undef SHL_FINISH
  return hipErrorInvalidValue;
}

hipError_t launch_pack(const PackList& l, hipStream_t s) {
  if (l.n == 0) return hipSuccess;
  const dim3 grid(pack_grid(l), l.n);
  if (l.f32)
    hipLaunchKernelGGL(pack_kernel<true>, grid, dim3(256), 0, s, l);
  else
    hipLaunchKernelGGL(pack_kernel<false>, grid, dim3(256), 0, s, l);
  return hipGetLastError();
}

}  // namespace shl
