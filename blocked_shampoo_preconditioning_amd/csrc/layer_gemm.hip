// The gated feed-forward block's products on the bf16 matrix cores.
//
// One tiled product serves the block's six: forward [g u] = x [Wg Wu] and
// y = h Wd; backward dh = dy Wd^T, dx = dg Wg^T + du Wu^T, [dWg dWu] = x^T [dg
// du] and dWd = h^T dy. Operands go from HBM to LDS without passing
// registers (buffer loads with an LDS destination, 16 bytes a lane), double
// buffered over K steps of 64; fragments leave LDS as 16-byte rows (K
// contiguous) or through the transposing 8-byte read (K the slow index), so no
// operand is ever transposed in memory.
#include "layer_device.h"
#include "layer_kernels.h"

namespace shl {

namespace {

typedef __attribute__((ext_vector_type(4))) int int4v;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short short4v;
typedef __attribute__((ext_vector_type(16))) float floatx16;
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kBK = 64;                 // K step
constexpr uint32_t kOutOfRange = 0x80000000u;

// ---------------------------------------------------------------- activation
__device__ __forceinline__ float sigmoidf(float x) { return 1.f / (1.f + __expf(-x)); }

// Value and derivative of the activation at g. The tanh form of GELU is
// g sigmoid(2 k (g + c g^3)), k = sqrt(2 / pi), c = 0.044715, since
// (1 + tanh(t)) / 2 = sigmoid(2 t).
__device__ __forceinline__ void activate(int act, float g, float& a, float& da) {
  if (act == kSilu) {
    const float s = sigmoidf(g);
    a = g * s;
    da = s * (1.f + g * (1.f - s));
  } else if (act == kGelu) {
    const float k = 0.7978845608028654f, c = 0.044715f;
    const float s = sigmoidf(2.f * k * g * (1.f + c * g * g));
    a = g * s;
    da = s + a * (1.f - s) * 2.f * k * (1.f + 3.f * c * g * g);
  } else {
    a = g > 0.f ? g : (g != g ? g : 0.f);
    da = g > 0.f ? 1.f : 0.f;
  }
}

// The epilogue on columns [col, col + 8) of one row: v (and for kGate also w,
// the same columns of u). Columns from N to pad_to get zeros.
template <int EPI>
__device__ __forceinline__ void finish8(const EpiArgs& e, int problem, int64_t row, int col, int N, float (&v)[8],
                                        float (&w)[8]) {
  const int width = e.pad_to > N ? e.pad_to : N;
  const int n = min(8, width - col);
  if (n <= 0) return;
  if (col + 8 > N) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i >= N) v[i] = 0.f, w[i] = 0.f;
  }
  const bool f32 = e.f32 != 0;
  if (EPI == kStore) {
    store8(problem ? e.c[1] : e.c[0], row * (problem ? e.ldc1 : e.ldc) + col, n, f32, v);
  } else if (EPI == kGate) {
    if (e.g) {
      store8(e.g, row * e.ldg + col, n, f32, v);
      store8(e.u, row * e.ldg + col, n, f32, w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      activate(e.act, v[i], a, da);
      v[i] = a * w[i];
    }
    store8(e.c[0], row * e.ldc + col, n, f32, v);
  } else {
    float g[8], u[8];
    load8(e.g, row * e.ldg + col, n, f32, g);
    load8(e.u, row * e.ldg + col, n, f32, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, da;
      activate(e.act, g[i], a, da);
      g[i] = v[i] * u[i] * da;
      u[i] = v[i] * a;
    }
    store8(e.c[0], row * e.ldc + col, n, f32, g);
    store8(e.c[1], row * e.ldc + col, n, f32, u);
  }
}

// ------------------------------------------------------------------ the tile
// WM x WN waves of FM x FN fragments of 32 x 32.
template <int FM_, int FN_, int WM_, int WN_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int BM = WM * FM * 32, BN = WN * FN * 32;
  static constexpr int A_BYTES = BM * kBK * 2, B_BYTES = BN * kBK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
};

// LDS order of 16-byte chunks. A row operand's tile is [rows][64 k] (8 chunks
// a row), a column operand's [64 k][width] (16 or 8 chunks a row). Chunk c of
// row r sits at place c ^ swizzle(r), so that the rows that one read takes
// together fall on different banks, whether the LDS serves 128 or 256 bytes
// at a time.
__device__ __forceinline__ int swz_row(int r) { return (r & 7) ^ ((r >> 3) & 1); }
template <int WIDTH>
__device__ __forceinline__ int swz_col(int k) {
  return WIDTH == 128 ? ((k & 3) << 1) ^ ((k & 3) << 2) : (k & 3) << 1;
}

// One panel of an operand on its way to LDS: `rows` rows of 128 (or WIDTH * 2)
// bytes, brought by all waves, 1 KiB an instruction.
struct Panel {
  const char* base;   // first byte of the panel at the current K step
  int64_t left;       // bytes from base to the operand's end
};

__device__ __forceinline__ int4v make_rsrc(const char* base, int64_t left) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  int64_t n = left < 0 ? 0 : (left + 3) & ~int64_t(3);
  n = n > 0x7ffffff0 ? 0x7ffffff0 : n;
  int4v r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(b >> 32) & 0xffff);
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(n));
  r[3] = 0x00020000;
  return r;
}

// 64 x 16 bytes from rsrc + voff (a lane's own) to LDS at `lds` + 16 * lane.
// Written as asm because the compiler would wait for every such load before
// any transposing LDS read; it has no register results, and its arrival is
// waited for at the barrier of the next K step.
__device__ __forceinline__ void load_lds(const int4v& rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "memory");
}

__device__ __forceinline__ bf16x8 lds_read16(const char* p) { return *reinterpret_cast<const bf16x8*>(p); }
__device__ __forceinline__ bf16x8 lds_read_tr(const char* p, int second) {
  typedef __attribute__((address_space(3))) short4v* P;
  union {
    short4v s[2];
    bf16x8 v;
  } x;
  x.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p));
  x.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + second));
  return x.v;
}

template <class T, bool ACOL, bool BCOL, int EPI>
__global__ __launch_bounds__(T::NT, T::NT == 512 ? 2 : 2) void gemm_kernel(GemmArgs g) {
  constexpr bool GATE = EPI == kGate;
  constexpr int HN = GATE ? T::BN / 2 : T::BN;       // result columns of a tile
  constexpr int AP = T::BM / 128;                    // A panels of 128 rows / columns
  constexpr int BW = GATE ? T::BN / 2 : 128;         // width of a B panel
  constexpr int BP = T::BN / BW;
  static_assert(BW == 128 || BW == 64, "");
  static_assert(!GATE || BCOL, "");
  __shared__ __attribute__((aligned(1024))) char lds[2 * T::STAGE];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM;

  // Workgroups go round the 8 XCDs; each XCD takes a contiguous range of the
  // work, in groups of four row tiles, so that the tiles in flight on one XCD
  // share their operands in its L2.
  const int tm = (g.M + T::BM - 1) / T::BM, tn = (g.N + HN - 1) / HN;
  const int64_t total = static_cast<int64_t>(tm) * tn * g.problems * g.splits;
  const int64_t per = (total + 7) / 8;
  int64_t id = static_cast<int64_t>(blockIdx.x % 8) * per + blockIdx.x / 8;
  if (id >= total || static_cast<int64_t>(blockIdx.x / 8) >= per) return;
  const int split = static_cast<int>(id / (static_cast<int64_t>(tm) * tn * g.problems));
  id -= static_cast<int64_t>(split) * tm * tn * g.problems;
  const int problem = static_cast<int>(id / (static_cast<int64_t>(tm) * tn));
  int t = static_cast<int>(id - static_cast<int64_t>(problem) * tm * tn);
  const int group = t / (4 * tn);
  const int in_group = min(4, tm - 4 * group);
  t -= group * 4 * tn;
  const int m0 = (4 * group + t % in_group) * T::BM, n0 = (t / in_group) * HN;

  // K steps of this split: segments of ksteps each
  const int ksteps = (g.K + kBK - 1) / kBK;
  const int steps = ksteps * g.nseg;
  const int first = static_cast<int>(static_cast<int64_t>(steps) * split / g.splits);
  const int last = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / g.splits);

  // a lane's place in the loads: offsets inside a panel, in bytes
  constexpr int A_INST = 16;                    // 1 KiB instructions of a 128-panel
  constexpr int B_INST = BW * kBK * 2 / 1024;
  const int64_t lda2 = g.lda * 2, ldb2 = g.ldb * 2;
  const uint32_t rsw = (lane & 7) ^ swz_row((lane >> 3) + 8 * wave);
  // rows a wave's instruction j covers: (j * NW + wave) * 8 (row operand) or * (1024 / row bytes)
  auto row_off = [&](int64_t ld2) { return static_cast<uint32_t>((wave * 8 + (lane >> 3)) * ld2 + rsw * 16); };
  auto col_off = [&](int64_t ld2, int width) {
    const int per_row = width / 8, rows = 64 / per_row;
    const int k = wave * rows + lane / per_row, p = lane % per_row;
    const int c = p ^ (width == 128 ? swz_col<128>(k) : swz_col<64>(k));
    return static_cast<uint32_t>(k * ld2 + c * 16);
  };
  const uint32_t a_off = ACOL ? col_off(lda2, 128) : row_off(lda2);
  const uint32_t b_off = BCOL ? col_off(ldb2, BW) : row_off(ldb2);
  const uint32_t a_jump = static_cast<uint32_t>((ACOL ? T::NW * 4 : T::NW * 8) * lda2);
  const uint32_t b_jump = static_cast<uint32_t>((BCOL ? T::NW * (512 / BW) : T::NW * 8) * ldb2);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char*)lds));

  auto issue = [&](int step, int buf) {
    const int seg = step / ksteps, k0 = (step - seg * ksteps) * kBK;
    const bool k_ok = k0 + static_cast<int>(rsw) * 8 < g.K;
    const uint32_t at = lds0 + buf * T::STAGE + wave * 1024;
#pragma unroll
    for (int p = 0; p < AP; ++p) {
      const char* base = reinterpret_cast<const char*>(g.a[seg]);
      const int64_t size = ACOL ? (static_cast<int64_t>(g.k_real) - 1) * lda2 + 2 * g.M
                                : (static_cast<int64_t>(g.M) - 1) * lda2 + 2 * g.K;
      const int64_t o = ACOL ? k0 * lda2 + 2 * (m0 + p * 128) : (m0 + p * 128) * lda2 + 2 * k0;
      const int4v rs = make_rsrc(base + o, size - o);
#pragma unroll
      for (int j = 0; j < A_INST / T::NW; ++j) {
        uint32_t v = a_off + j * a_jump;
        if (!ACOL) v = k_ok ? v : kOutOfRange;
        load_lds(rs, v, at + p * 16384 + j * T::NW * 1024);
      }
    }
#pragma unroll
    for (int p = 0; p < BP; ++p) {
      const char* base = reinterpret_cast<const char*>(GATE ? g.b[p][seg] : g.b[problem][seg]);
      const int64_t size = BCOL ? (static_cast<int64_t>(g.k_real) - 1) * ldb2 + 2 * g.N
                                : (static_cast<int64_t>(g.N) - 1) * ldb2 + 2 * g.K;
      const int col = n0 + (GATE ? 0 : p * 128);
      const int64_t o = BCOL ? k0 * ldb2 + 2 * col : col * ldb2 + 2 * k0;
      const int4v rs = make_rsrc(base + o, size - o);
#pragma unroll
      for (int j = 0; j < B_INST / T::NW; ++j) {
        uint32_t v = b_off + j * b_jump;
        if (!BCOL) v = k_ok ? v : kOutOfRange;
        load_lds(rs, v, at + T::A_BYTES + p * (B_INST * 1024) + j * T::NW * 1024);
      }
    }
  };

  // a lane's place in the fragment reads
  const int half = lane >> 5, r32 = lane & 31;
  // row operand: row r32 of a fragment, chunk 2 ks + half
  auto frag_row = [&](const char* tile, int row0, int ks) {
    return lds_read16(tile + (row0 + r32) * 128 + (((2 * ks + half) ^ swz_row(r32)) << 4));
  };
  // column operand: k = 16 ks + 8 half + (lane % 16) / 4 (+ 4 in the second
  // read), columns 16 ((lane / 16) % 2) + 4 (lane % 4)
  const int kk = (lane & 15) >> 2;
  auto frag_col = [&](const char* tile, int width, int col0, int ks) {
    const int c = (col0 >> 3) + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int s = width == 128 ? swz_col<128>(kk) : swz_col<64>(kk);
    const char* p = tile + (16 * ks + 8 * half + kk) * (width * 2) + ((c ^ s) << 4) + (lane & 1) * 8;
    return lds_read_tr(p, 4 * width * 2);
  };
  auto frag_a = [&](const char* st, int i, int ks) {
    const int row = wm * T::FM * 32 + i * 32;  // within the tile
    if (ACOL) return frag_col(st + (row >> 7) * 16384, 128, row & 127, ks);
    return frag_row(st, row, ks);
  };
  auto frag_b = [&](const char* st, int j, int ks) {
    const char* bt = st + T::A_BYTES;
    if (GATE) {  // even fragments: gate panel, odd: up panel
      const int col = wn * (T::FN / 2) * 32 + (j >> 1) * 32;
      return frag_col(bt + (j & 1) * (B_INST * 1024), BW, col, ks);
    }
    const int col = wn * T::FN * 32 + j * 32;
    if (BCOL) return frag_col(bt + (col >> 7) * 16384, 128, col & 127, ks);
    return frag_row(bt, col, ks);
  };

  floatx16 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  if (first < last) issue(first, 0);
  for (int step = first; step < last; ++step) {
    const int buf = (step - first) & 1;
    // this wave's loads of the step have landed and its reads of the other
    // buffer are done; after the barrier that holds for all waves
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (step + 1 < last) issue(step + 1, buf ^ 1);
    const char* st = lds + buf * T::STAGE;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8 a[T::FM], b[T::FN];
#pragma unroll
      for (int i = 0; i < T::FM; ++i) a[i] = frag_a(st, i, ks);
#pragma unroll
      for (int j = 0; j < T::FN; ++j) b[j] = frag_b(st, j, ks);
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // Epilogue. A lane's accumulators are column r32 (row m of the result) and
  // rows 8 q + 4 half + 0..3 (result columns n) of each fragment: FN fragments
  // pass through a wave-private LDS strip and come back as eight columns of
  // one row a lane, so that stores are 16 bytes a lane and whole row segments.
  constexpr int PITCH = T::FN * 32 + 4;
  float* strip = reinterpret_cast<float*>(lds) + wave * (32 * PITCH);
  static_assert(T::NW * 32 * PITCH * 4 <= 2 * T::STAGE, "");
  const EpiArgs& e = g.e;
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        floatx4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = acc[i][j][4 * q + r];
        *reinterpret_cast<floatx4*>(strip + r32 * PITCH + j * 32 + 8 * q + 4 * half) = x;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int COLS = GATE ? T::FN * 16 : T::FN * 32;   // result columns of a wave
    constexpr int LR = COLS / 8, RP = 64 / LR;             // lanes a row, rows a pass
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += RP) {
      const int r = r0 + lane / LR, c8 = (lane % LR) * 8;
      const int64_t row = m0 + wm * T::FM * 32 + i * 32 + r;
      const int col = n0 + wn * COLS + c8;
      float v[8], w[8];
      if (GATE) {
        const float* p = strip + r * PITCH + (c8 >> 5) * 64 + (c8 & 31);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = p[q], w[q] = p[32 + q];
      } else {
        const float* p = strip + r * PITCH + c8;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = p[q], w[q] = 0.f;
      }
      if (row < g.M) {
        if (g.splits > 1) {
          constexpr int parts = GATE ? 2 : 1;
          const int n = min(8, g.N - col);
          float* q = g.partial + ((static_cast<int64_t>(split) * g.problems + problem) * parts) * g.M * g.N + row * g.N + col;
          if (n > 0) {
            store8(q, 0, n, true, v);
            if (GATE) store8(q + static_cast<int64_t>(g.M) * g.N, 0, n, true, w);
          }
        } else {
          finish8<EPI>(e, problem, row, col, g.N, v, w);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Joins the parts of a split product in their order and runs the epilogue.
template <int EPI>
__global__ __launch_bounds__(256) void gemm_finish_kernel(GemmArgs g) {
  const int width = max(g.N, g.e.pad_to);
  const int c8 = (width + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(c8) * g.M) return;
  const int problem = blockIdx.y;
  const int64_t row = i / c8;
  const int col = static_cast<int>(i - row * c8) * 8;
  constexpr int parts = EPI == kGate ? 2 : 1;
  const int64_t plane = static_cast<int64_t>(g.M) * g.N;
  const int n = max(0, min(8, g.N - col));
  float v[8], w[8], x[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = w[q] = 0.f;
  for (int s = 0; s < g.splits; ++s) {
    const float* p = g.partial + (static_cast<int64_t>(s) * g.problems + problem) * parts * plane + row * g.N + col;
    load8(p, 0, n, true, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += x[q];
    if (EPI == kGate) {
      load8(p + plane, 0, n, true, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] += x[q];
    }
  }
  finish8<EPI>(g.e, problem, row, col, g.N, v, w);
}

// ------------------------------------------------------------------- packing
// x = h + m + l exactly, each term bf16: h and m by cutting the low 16 bits,
// l what is left (at most 8 significant bits). Infinities and NaN stay in h.
__global__ __launch_bounds__(256) void pack_planes_kernel(PackArgs p) {
  const int64_t c8 = p.ld_out / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= c8 * p.rows) return;
  const int64_t row = i / c8;
  const int col = static_cast<int>(i - row * c8) * 8;
  const int n = static_cast<int>(p.cols - col < 8 ? (p.cols - col < 0 ? 0 : p.cols - col) : 8);
  float v[8];
  load8(p.src, row * p.ld + col, n, p.f32 != 0, v);
  const int64_t at = row * p.ld_out + col, plane = p.rows * p.ld_out;
  uint4v h, m, l;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t t[2][3];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float x = v[2 * q + b];
      const float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      float d = x - hx;
      if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) d = 0.f;
      const float mx = __uint_as_float(__float_as_uint(d) & 0xffff0000u);
      // a NaN whose payload lies in the low bits only stays a NaN
      t[b][0] = (__float_as_uint(hx) >> 16) | ((x != x) ? 0x40u : 0u);
      t[b][1] = __float_as_uint(mx) >> 16;
      t[b][2] = __float_as_uint(d - mx) >> 16;
    }
    h[q] = t[0][0] | t[1][0] << 16;
    m[q] = t[0][1] | t[1][1] << 16;
    l[q] = t[0][2] | t[1][2] << 16;
  }
  *reinterpret_cast<uint4v*>(p.out + at) = h;
  if (p.f32) {
    *reinterpret_cast<uint4v*>(p.out + plane + at) = m;
    *reinterpret_cast<uint4v*>(p.out + 2 * plane + at) = l;
  }
}

using Tile256 = Tile<4, 2, 2, 4>;
using Tile128 = Tile<2, 2, 2, 2>;

template <class T, bool ACOL, bool BCOL, int EPI>
hipError_t launch_one(const GemmArgs& g, hipStream_t s) {
  const int64_t tiles = gemm_tiles(g.M, g.N, g.problems, T::BM, EPI == kGate) * g.splits;
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_kernel<T, ACOL, BCOL, EPI>), dim3(static_cast<uint32_t>(grid)), dim3(T::NT), 0, s, g);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || g.splits == 1) return err;
  const int64_t c8 = (((g.e.pad_to > g.N) ? g.e.pad_to : g.N) + 7) / 8;
  const int64_t blocks = (c8 * g.M + 255) / 256;
  hipLaunchKernelGGL((gemm_finish_kernel<EPI>), dim3(static_cast<uint32_t>(blocks), g.problems), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace

int64_t gemm_tiles(int64_t M, int64_t N, int problems, int tile, bool gate) {
  const int64_t hn = gate ? tile / 2 : tile;
  return ((M + tile - 1) / tile) * ((N + hn - 1) / hn) * problems;
}

int64_t gemm_steps(int64_t K, int nseg) { return (K + kBK - 1) / kBK * nseg; }

hipError_t launch_gemm(const GemmArgs& g, int tile, bool a_cols, bool b_cols, Epi epi, hipStream_t s) {
  if (g.M <= 0 || g.N <= 0) return hipSuccess;
#define SHL_CASE(AC, BC, E)                                              \
  if (a_cols == AC && b_cols == BC && epi == E)                          \
    return tile == 256 ? launch_one<Tile256, AC, BC, E>(g, s) : launch_one<Tile128, AC, BC, E>(g, s);
  SHL_CASE(false, true, kGate)
  SHL_CASE(false, true, kStore)
  SHL_CASE(false, false, kActBwd)
  SHL_CASE(false, false, kStore)
  SHL_CASE(true, true, kStore)
#undef SHL_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_pack(const PackArgs& p, hipStream_t s) {
  const int64_t n = p.rows * (p.ld_out / 8);
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(pack_planes_kernel, dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace shl
