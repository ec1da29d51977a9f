// Launchers of the experts' kernels (experts_route.hip, experts_quantize.hip,
// experts_product.hip, experts_few.hip), called by the host side
// of the C ABI (experts_runtime.cpp). Not public.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace she {

struct SortArgs {
  const void* ids;
  int64_t ld_ids;
  uint32_t slots, total, experts;  // total = tokens * slots
  uint32_t per_block;              // slot numbers of a workgroup
  uint32_t blocks;
  int32_t wide;                    // 64-bit ids
  int32_t *offsets, *rows, *source;
  uint32_t* counts;                // [blocks][experts + 1], blocks > 1
};
// Workgroups and slot numbers of each for `total` slots.
void sort_plan(int64_t total, uint32_t& blocks, uint32_t& per_block);
hipError_t launch_sort(const SortArgs& a, hipStream_t s);

struct RouteArgs {
  int64_t tokens;
  uint32_t slots, total;  // total = tokens * slots
  int32_t width, f32;
  const int32_t* rows;
  const float* weights;
  const void *x, *ys;
  int64_t ld_x, ld_ys;
  void *y, *xs;
  int64_t ld_y, ld_xs;
  float* dweights;
  bool past;  // xs is written past the caches
};
hipError_t launch_dispatch(const RouteArgs& a, hipStream_t s);
hipError_t launch_combine(const RouteArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const RouteArgs& a, hipStream_t s);

// ------------------------------------------------------ 8-bit products
// Values in 8 bits are e4m3, their scales exponents with a bias of 127. An
// operand of a product has its rows along its summation index, K: bytes
// [rows][K rounded up to 128], zero behind K. Rows of tokens come in blocks of
// 128 that begin with each expert's first row ("padded rows"), so that a block is
// one expert's and the scales of a token block are one expert's too.
constexpr int kBlock = 128;

// Where row (or column) i of a block of 128 has its scale: the matrix
// instruction's operand i / 16 of a lane takes rows that make a lane's results
// 16 consecutive columns, and a lane reads the scales of its eight rows at once.
__host__ __device__ constexpr int scale_place(int i) { return (((i >> 4) & 3) * 4 + (i & 3)) * 8 + (i >> 6) * 4 + ((i >> 2) & 3); }
// The row of operand f of 16 rows, row r of it.
__host__ __device__ constexpr int operand_row(int f, int r) { return 64 * (f >> 2) + 16 * (r >> 2) + 4 * (f & 3) + (r & 3); }

// The experts' rows: expert e has offsets[e] .. offsets[e + 1] of n (offsets
// NULL: one expert has all).
struct Groups {
  const int32_t* offsets;
  int32_t n, experts;
  int32_t blocks;  // at least as many as all experts' rows take
};

// C = sum over k of A[m][k] B[n][k] with their scales, on the matrix cores.
// by_expert 0: rows of tokens against one matrix an expert (y, dx), rows behind the
// last expert's get 0. 1: for each expert, over its blocks of padded rows (dW).
struct ProductArgs {
  const uint8_t *a, *a_scales, *b, *b_scales;
  int64_t pitch;                     // bytes of a row of a and b
  int64_t size_a, size_b;            // bytes; of b, one expert's
  int64_t b_stride, b_scale_stride;  // from an expert to the next
  int32_t a_blocks, b_blocks;        // of 128 rows: the scales' [K block][blocks][128], or b's [blocks][b_scale_pitch]
  int32_t b_scale_pitch;
  int32_t M, N, k_blocks;
  int32_t by_expert;
  void* c;
  int64_t ldc, c_stride;
};
// Rows and columns of a result tile; fp32 results have kProduct128 alone.
// kProduct128Deep: one workgroup a CU with four steps' operands in LDS, for few tiles.
enum ProductTile { kProduct256, kProduct128, kProduct128Deep };
constexpr int product_tile(ProductTile t) { return t == kProduct256 ? 256 : 128; }
// One or two products in one launch, of one type. Their work, a record for each
// tile, is written by the launch that quantizes an operand: who has which rows is on
// the GPU, and a workgroup that worked out its tile itself would wait for it in front
// of its first loads (measured: 5 us of a launch).
constexpr int kMaxProducts = 2;
struct WorkRecord {
  uint64_t a, b;              // addresses of the tile's first row and K block
  uint32_t size_a, size_b;    // bytes from there on (at most 2^32 - 16)
  uint64_t a_scales, b_scales;
  uint32_t a_scales_size, b_scales_size;
  uint64_t c;
  int32_t turns;              // K blocks; < 0: no tile, see below
  uint32_t shape;             // rows, columns << 10, words << 20, second << 21, product << 22
};
static_assert(sizeof(WorkRecord) == 64, "");
constexpr int kNoTile = -1, kNoTileNorBehind = -2;
struct Products {
  ProductArgs p[kMaxProducts];
  int32_t count, experts, f32;
  WorkRecord* work;  // [8][per]: an XCD's tiles in order
  int32_t per;
  int32_t tile;      // ProductTile
};
// Tiles an XCD can have at most, for Products::per.
int64_t work_length(const Products& a, int64_t rows, bool grouped);
hipError_t launch_products(const Products& a, hipStream_t s);

// 128 x 128 tiles of x in 8 bits: by rows (a scale for each row of the tile), by
// columns (a scale for each column, values transposed), either or both; and the
// records of the products' work.
struct QuantizeArgs {
  const void* x;
  int64_t ld;
  int32_t f32, cols, col_blocks;
  Groups g;
  const int32_t* source;  // padded row r of x is row source[r] / slots; NULL: r
  uint32_t slots;
  int32_t rows_in;        // rows of x
  // not NULL, and by rows alone: tiles are of x, and each row's values go to the
  // padded rows of its slots' rows [rows_in][slots]
  const int32_t* slot_rows;
  uint8_t *by_rows, *row_scales;  // [128 blocks][128 col_blocks], [col_blocks][blocks][128]
  uint8_t *by_cols, *col_scales;  // [128 col_blocks][128 blocks], [blocks][col_blocks][128]
  Products products;
};
constexpr int kMaxScatter = 16;  // slots with slot_rows
hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s);

// Weights w [in][out], one scale for each tile: transposed ("forward": [out][in])
// and as they lie ("backward": [in][out]), rows padded to 128, scale rows to 4.
struct WeightArgs {
  const void* w;
  int64_t ld, expert_stride;
  int32_t f32, experts, in, out;
  uint8_t *forward, *forward_scales, *backward, *backward_scales;
};
hipError_t launch_quantize_weight(const WeightArgs& a, hipStream_t s);

// Rows of tokens, 64 at most in all, against one matrix an expert, in one launch:
// x is quantized as it is read.
constexpr int kFewRows = 64;
struct FewArgs {
  const void* x;
  int64_t ld_x;
  Groups g;                // blocks is not read
  const int32_t* source;
  uint32_t slots;
  int32_t rows_in;
  const uint8_t *b, *b_scales;
  int64_t pitch_b, b_stride, b_scale_stride;
  int32_t b_scale_pitch;
  int32_t K, N;
  void* c;
  int64_t ldc;
  int32_t f32;
};
hipError_t launch_few(const FewArgs& a, hipStream_t s);

}  // namespace she
