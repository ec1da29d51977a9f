// The feed-forward block's forward products for a few tokens (serving).
//
// Every weight is read once for at most 16 T rows of x, so HBM sets the floor; the
// kernel reads at 3.4 TB/s where a copy reaches 5.3. What it asks for is what it
// needs (misses of the L2s: the weights' own bytes), but in pieces of half a
// cache line (half of the L2s' requests are hits on the other half), and small
// weights make fewer workgroups than the card has CUs (13 tokens of 768 x 2048: 64
// and 96). The weights' rows [k][n] go from memory into registers, two columns a
// lane: the 16 lanes of a row read 32 columns in whole 64-byte pieces, and
// each wave has 8 to 16 loads a matrix in flight with no LDS in their way. The
// matrix cores take them as they come: the weights are the "A" operand (16 rows
// of one 16 x 16 product are columns 2 j + i, j the lane of a row), x the "B"
// operand (16 tokens). fp32 uses the fp32 matrix instruction, so it is exact to
// fp32 accumulation. bf16 h comes as two bf16 terms: its rounding would save no
// weight byte, and y is off by 0.0024 in norm with one term, by its own rounding,
// 0.0017, with two (16 tokens of 2048 x 8192 35.7 and 39.1 us, 32 43 and 46).
//
// One token of 2048 x 8192 bf16: g, u and h (67 MB) in 20 us, y (34 MB) in 10 and
// 4 to join its 8 parts of K (16 and 8 for the products when the last-level
// cache still has the weights); 13 tokens of 768 x 2048 fp32 (19 MB): 10, 5 and 3,
// where the launches are more than half; 64 tokens of 2048 x 8192 fp32 (201 MB) in
// 105. Loaded as one batch of 64 rows at a time: 33.5 us against 32.4 for the
// one token, 120 against 105 for the 64. Two batches of 64 spill; non-temporal
// loads are no faster.
#include "layer_epilogue.h"
#include "layer_kernels.h"

namespace shl {

namespace {

typedef __attribute__((ext_vector_type(4))) short short4v;

constexpr int kCols = 32;       // columns of a workgroup
constexpr int kBatch = 32;      // K rows of a load; a wave has one or two of them in flight
constexpr int kRun = kBatch / 4;  // the run of them that a lane has

// A batch's K rows go to the 16-lane groups q = 0..3 in runs of kRun, so that a
// lane's values of x lie together: step s of the products takes row kRun q + s
// (fp32, four rows a product) or rows kRun q + 4 s + 0..3 (bf16, sixteen).
//
// kRun values of x of one token; those from K on are zeros.
template <bool F32>
constexpr int kWords = F32 ? kRun : kRun / 2;
template <bool F32>
__device__ __forceinline__ void load_x(const void* x, int64_t row, int k, int K, uint32_t (&v)[kWords<F32>]) {
  if (k + kRun <= K) {
    __builtin_memcpy(v, static_cast<const char*>(x) + (row + k) * (F32 ? 4 : 2), 4 * kWords<F32>);
    return;
  }
#pragma unroll
  for (int i = 0; i < kWords<F32>; ++i) v[i] = 0;
#pragma unroll 1
  for (int e = K - k - 1; e >= 0; --e) {  // shifted in from the last one
#pragma unroll
    for (int i = kWords<F32> - 1; i > 0; --i) v[i] = F32 ? v[i - 1] : v[i] << 16 | v[i - 1] >> 16;
    if constexpr (F32)
      v[0] = static_cast<const uint32_t*>(x)[row + k + e];
    else
      v[0] = v[0] << 16 | static_cast<const uint16_t*>(x)[row + k + e];
  }
}

// A lane's first column, at most that of the last pair. bf16 pairs are aligned
// words, so of an odd N the last one has the next row's element, or a pad, in its
// second place (the buffer's length is rounded up to a word for the last row's);
// fp32 pairs end with the last column.
template <bool F32>
__device__ __forceinline__ int pair_col(int n, int N) {
  return min(n, F32 ? N - 2 : (N - 1) & ~1);
}

// kBatch rows of K from k0 for MATS matrices and 16 T tokens. Rows from K on lie
// past the weights' end and read as zeros; what a lane reads past a row's last
// column belongs to columns that are not stored.
template <bool F32, int MATS, int T, int TERMS>
struct Batch {
  uint32_t w[MATS][kRun][F32 ? 2 : 1], x[TERMS][T][kWords<F32>];
};
template <bool F32, int MATS, int T, int TERMS>
__device__ __forceinline__ void load(const DecodeArgs& a, const int64_t (&xrow)[T], int k0, const uint32_t (&off)[MATS],
                                     Batch<F32, MATS, T, TERMS>& b) {
  constexpr int E = F32 ? 4 : 2;
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    load_x<F32>(a.x, xrow[t], k0 + kRun * q, a.K, b.x[0][t]);
    if constexpr (TERMS == 2) load_x<F32>(a.x_rest, xrow[t], k0 + kRun * q, a.K, b.x[1][t]);
  }
#pragma unroll
  for (int m = 0; m < MATS; ++m) {
    const int64_t at = k0 * a.ldw[m] * E, end = (((a.K - 1) * a.ldw[m] + a.N) * E + 3) & ~int64_t(3);
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(a.w[m]) + at), 0, static_cast<int>(max<int64_t>(0, min<int64_t>(end - at, 0x7ffffff0))), 0x00020000);
    const uint32_t step = static_cast<uint32_t>(a.ldw[m]) * E;
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
      if constexpr (F32) {
        typedef __attribute__((ext_vector_type(2))) uint32_t uint2v;
        const uint2v w = __builtin_bit_cast(uint2v, __builtin_amdgcn_raw_buffer_load_b64(r, off[m] + s * step, 0, 0));
        b.w[m][s][0] = w[0], b.w[m][s][1] = w[1];
      } else {
        b.w[m][s][0] = __builtin_amdgcn_raw_buffer_load_b32(r, off[m] + s * step, 0, 0);
      }
    }
  }
}

// Their products.
template <bool F32, int MATS, int T, int TERMS>
__device__ __forceinline__ void use(const Batch<F32, MATS, T, TERMS>& b, floatx4 (&acc)[MATS][2][T]) {
  if constexpr (F32) {
#pragma unroll
    for (int s = 0; s < kRun; ++s)
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int t = 0; t < T; ++t)
            acc[m][i][t] =
                __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b.w[m][s][i]), __uint_as_float(b.x[0][t][s]), acc[m][i][t], 0, 0, 0);
  } else {
    typedef __attribute__((ext_vector_type(2))) uint32_t uint2v;
#pragma unroll
    for (int s = 0; s < kRun / 4; ++s)
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const uint32_t w0 = b.w[m][4 * s][0], w1 = b.w[m][4 * s + 1][0], w2 = b.w[m][4 * s + 2][0], w3 = b.w[m][4 * s + 3][0];
        // four rows of the lane's first and second column
        const uint2v c0 = {__builtin_amdgcn_perm(w1, w0, 0x05040100u), __builtin_amdgcn_perm(w3, w2, 0x05040100u)};
        const uint2v c1 = {__builtin_amdgcn_perm(w1, w0, 0x07060302u), __builtin_amdgcn_perm(w3, w2, 0x07060302u)};
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e) {
            const uint2v xx = {b.x[e][t][2 * s], b.x[e][t][2 * s + 1]};
            const short4v x4 = __builtin_bit_cast(short4v, xx);
            acc[m][0][t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4v, c0), x4, acc[m][0][t], 0, 0, 0);
            acc[m][1][t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4v, c1), x4, acc[m][1][t], 0, 0, 0);
          }
        }
      }
  }
}

// Workgroup: kCols columns (of both weights for kGate), one of a.splits parts
// of K, cut again over the waves; the waves' sums are added in order through
// LDS. One part: the epilogue follows; more: the sums go to a.partial in
// GemmArgs' layout and the finish kernel joins them.
//
// The second term of x (TERMS = 2, or FOLD: at most eight tokens, whose second
// terms take the place of tokens 8 to 15) has its sums added to the first's.
// Folded, one token of 2048 x 8192 takes 32.5 us, with one term 32.3; with twice the
// registers for x 34.1, since they leave room for one workgroup of 16 waves on a
// CU in place of two.
template <bool F32, int EPI, int T, int W, int TERMS>
__global__ __launch_bounds__(W * 64) void decode_kernel(DecodeArgs a) {
  constexpr int MATS = EPI == kGate ? 2 : 1;
  constexpr bool FOLD = !F32 && EPI == kStore && TERMS == 1;
  static_assert(!FOLD || T == 1, "");
  constexpr int PITCH = kCols + 4;
  __shared__ float sums[W][MATS * 16][PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring columns, whose rows share cache lines, go to one XCD
  const uint32_t per = gridDim.x / 8;
  const uint32_t id = blockIdx.x % 8 * per + blockIdx.x / 8;
  const uint32_t groups = (a.N + kCols - 1) / kCols;
  if (id >= groups * a.splits) return;
  const uint32_t group = id / a.splits, split = id - group * a.splits;
  // a lane's two columns; the last lanes repeat the matrix's last pair
  const int n0 = group * kCols, col = pair_col<F32>(n0 + 2 * (lane & 15), a.N);
  uint32_t off[MATS];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
    off[m] = (kRun * (lane >> 4) * static_cast<uint32_t>(a.ldw[m]) + static_cast<uint32_t>(col)) * (F32 ? 4 : 2);
  // batches of this wave
  const int batches = (a.K + kBatch - 1) / kBatch, parts = a.splits * W;
  const int part = split * W + wave, each = batches / parts, rest = batches - each * parts;
  const int first = each * part + min(part, rest), last = first + each + (part < rest ? 1 : 0);
  int64_t xrow[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    xrow[t] = static_cast<int64_t>(min(16 * t + (lane & (FOLD ? 7 : 15)), a.M - 1)) * a.ldx;
    if (FOLD && (lane & 8)) xrow[t] += static_cast<const uint16_t*>(a.x_rest) - static_cast<const uint16_t*>(a.x);
  }
  floatx4 acc[MATS][2][T];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[m][i][t] = floatx4{0.f, 0.f, 0.f, 0.f};
  // one batch is loaded while the one before it is multiplied
  Batch<F32, MATS, T, TERMS> even, odd;
  int b = first;
  if (b < last) load<F32, MATS, T, TERMS>(a, xrow, b * kBatch, off, even);
#pragma unroll 1
  for (; b + 2 < last; b += 2) {
    load<F32, MATS, T, TERMS>(a, xrow, (b + 1) * kBatch, off, odd);
    use<F32, MATS, T, TERMS>(even, acc);
    load<F32, MATS, T, TERMS>(a, xrow, (b + 2) * kBatch, off, even);
    use<F32, MATS, T, TERMS>(odd, acc);
  }
  if (b + 1 < last) load<F32, MATS, T, TERMS>(a, xrow, (b + 1) * kBatch, off, odd);
  if (b < last) use<F32, MATS, T, TERMS>(even, acc);
  if (b + 1 < last) use<F32, MATS, T, TERMS>(odd, acc);
  const Activation<F32> act(a.e.act);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int rows = min(16, a.M - 16 * t);
    if (rows <= 0) break;
    if (t > 0) __syncthreads();
    // a lane's sums: token lane % 16, columns of the lanes 4 (lane / 16) + r
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = pair_col<F32>(n0 + 2 * (4 * (lane >> 4) + r), a.N) + i - n0;
        if (c >= 0) {
#pragma unroll
          for (int m = 0; m < MATS; ++m) sums[wave][m * 16 + (lane & 15)][c] = acc[m][i][t][r];
        }
      }
    __syncthreads();
    // the waves' sums in order, one column of one token a lane
#pragma unroll 1
    for (int u = threadIdx.x; u < MATS * rows * kCols; u += W * 64) {
      const int c = u % kCols, y = u / kCols, row = y < rows ? y : y - rows + 16;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) x += FOLD ? sums[k][row][c] + sums[k][row + 8][c] : sums[k][row][c];
      sums[0][row][c] = x;
    }
    __syncthreads();
#pragma unroll 1
    for (int u = threadIdx.x; u < rows * (kCols / 8); u += W * 64) {
      const int row = u / (kCols / 8), c = u % (kCols / 8) * 8, token = 16 * t + row;
      float v[8], w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = sums[0][row][c + q];
        w[q] = MATS == 2 ? sums[0][(MATS - 1) * 16 + row][c + q] : 0.f;
      }
      if (a.splits > 1) {
        const int n = min(8, a.N - n0 - c);
        const int64_t plane = static_cast<int64_t>(a.M) * a.N;
        float* p = a.partial + static_cast<int64_t>(split) * MATS * plane + static_cast<int64_t>(token) * a.N + n0 + c;
        if (n > 0) {
          store8(p, 0, n, true, v);
          if (MATS == 2) store8(p + plane, 0, n, true, w);
        }
      } else {
        const Raw8<F32> none{};
        finish8<F32, EPI>(a.e, act, 0, token * a.e.ldc + n0 + c, token * a.e.ldg + n0 + c, n0 + c, a.N, v, w, none, none);
      }
    }
  }
}

template <bool F32, int EPI>
hipError_t launch_decode_tokens(const DecodeArgs& a, dim3 grid, hipStream_t s) {
  constexpr int TERMS = !F32 && EPI == kStore ? 2 : 1;
  // more tokens take more registers a wave, so fewer waves
  if (a.M <= 8)
    hipLaunchKernelGGL((decode_kernel<F32, EPI, 1, F32 ? 8 : 16, 1>), grid, dim3(F32 ? 512 : 1024), 0, s, a);
  else if (a.M <= 16)
    hipLaunchKernelGGL((decode_kernel<F32, EPI, 1, F32 ? 8 : 16, TERMS>), grid, dim3(F32 ? 512 : 1024), 0, s, a);
  else if (a.M <= 32)
    hipLaunchKernelGGL((decode_kernel<F32, EPI, 2, 8, TERMS>), grid, dim3(512), 0, s, a);
  else if constexpr (F32)
    hipLaunchKernelGGL((decode_kernel<F32, EPI, 4, 8, TERMS>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t decode_groups(int64_t N) { return (N + kCols - 1) / kCols; }
int64_t decode_batches(int64_t K) { return (K + kBatch - 1) / kBatch; }

hipError_t launch_decode(const DecodeArgs& a, bool f32, Epi epi, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  if (a.M > decode_tokens(f32) || (epi != kGate && epi != kStore)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>((decode_groups(a.N) * a.splits + 7) / 8 * 8));
  hipError_t e;
  if (epi == kGate)
    e = f32 ? launch_decode_tokens<true, kGate>(a, grid, s) : launch_decode_tokens<false, kGate>(a, grid, s);
  else
    e = f32 ? launch_decode_tokens<true, kStore>(a, grid, s) : launch_decode_tokens<false, kStore>(a, grid, s);
  if (e != hipSuccess || a.splits == 1) return e;
  GemmArgs g{};
  g.M = a.M, g.N = a.N, g.problems = 1, g.splits = a.splits, g.partial = a.partial, g.e = a.e, g.f32 = f32;
  return launch_finish(g, epi, s);
}

}  // namespace shl
