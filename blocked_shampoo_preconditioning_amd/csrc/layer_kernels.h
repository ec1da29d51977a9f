// Launchers of the layer operators' kernels (layer_gemm.hip, layer_norm.hip),
// called by the host side of the C ABI (layer_runtime.cpp). Not public.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace shl {

constexpr int kMaxSeg = 2;  // the gradient of x is the sum of two products
// bf16 terms of an operand: fp32 values are the sum of three (split3)
constexpr int planes(bool f32) { return f32 ? 3 : 1; }

enum Act { kSilu = 0, kGelu = 1, kRelu = 2 };

// What happens to a finished tile of the product.
enum Epi {
  kStore = 0,   // C = acc
  kGate = 1,    // two products g, u side by side: h = act(g) u (g, u stored for training)
  kActBwd = 2   // acc = dh: dg = dh u act'(g), du = dh act(g)
};

struct EpiArgs {
  void* c[2];          // kStore: results of problems 0, 1; kGate: h, and in bf16 (may be NULL)
                       // what its rounding leaves; kActBwd: dg, du
  void* g;             // kGate: stores of g, u (NULL: not kept); kActBwd: loads
  void* u;
  int64_t ldc, ldc1;   // elements; ldc1: problem 1's (kStore)
  int64_t ldg;
  int32_t act;
  int32_t pad_to;      // columns [N, pad_to) are written as zeros (rows padded for a later product)
  int64_t plane;       // f32, kGate and kActBwd: c are planes, `plane` elements apart; 0: fp32 arrays
};

// sum over segments s of A_s B_s, A_s [M][K], B_s [K][N], bf16 operands with
// fp32 accumulation. An operand is read by rows (K contiguous) or by columns (K
// is the slow index). f32 = 0: bf16 operands and bf16 arrays in the epilogue; 1:
// operands are three bf16 planes whose sum is the fp32 value, arrays fp32.
struct GemmArgs {
  const uint16_t* a[kMaxSeg];
  const uint16_t* b[2][kMaxSeg];  // [1]: u's weights (kGate) or problem 1's operand
  int64_t lda, ldb;
  int64_t plane_a, plane_b;       // f32: elements from one plane to the next
  int32_t f32;
  int32_t nseg;
  int32_t M, N;        // N: columns of one result
  int32_t K;           // a multiple of 8: rows of a row operand are whole 16-byte chunks
  int32_t k_real;      // rows of a column operand (the rest of K reads as zero)
  int32_t problems;    // 1 or 2 (same A, other B and C)
  int32_t splits;      // the K range is cut in this many parts, joined by the finish kernel
  float* partial;      // [splits][problems * parts][M][N], splits > 1
  EpiArgs e;
};

// Results of a workgroup: 256 x 256, 128 x 128 or 128 x 256 (kGate: 128 or 64
// columns of h); x2: by two sets of waves with half of K each. bf16 takes the
// first three, f32 kTile128 and kTileWide.
enum TileKind { kTile256, kTile128, kTile128x2, kTileWide };
constexpr bool is_tile(TileKind t, bool f32) { return f32 ? t == kTile128 || t == kTileWide : t != kTileWide; }
hipError_t launch_gemm(const GemmArgs& g, TileKind tile, bool a_cols, bool b_cols, Epi epi, hipStream_t s);
// Tiles of one launch before splitting.
int64_t gemm_tiles(int64_t M, int64_t N, int problems, TileKind tile, bool gate);
// K steps of one launch (all segments): of 64, f32 of 32 (which has six products).
int64_t gemm_steps(int64_t K, int nseg, bool f32);

// Three products of one launch: g[0] reads both operands by rows, g[1] and g[2]
// by columns; all store (M = 0: left out). start is filled by the launch.
struct GroupArgs {
  GemmArgs g[3];
  uint32_t start[4];
};
hipError_t launch_group(GroupArgs& a, TileKind tile, bool f32, hipStream_t s);
// Joins a split product's parts and runs the epilogue.
hipError_t launch_finish(const GemmArgs& g, Epi epi, hipStream_t s);

// A forward product for at most decode_tokens rows of x: x [M][K], w [K][N] (kGate: both weights), bf16 weights with 4-byte
// aligned rows; K, N >= 2.
constexpr int decode_tokens(bool f32) { return f32 ? 64 : 32; }
struct DecodeArgs {
  const void* x;
  const void* x_rest;  // bf16, kStore: the second term of x (same layout)
  const void* w[2];
  int64_t ldx, ldw[2];
  int32_t M, N, K, splits;
  float* partial;      // [splits][1 or 2][M][N], splits > 1
  EpiArgs e;
};
int64_t decode_groups(int64_t N);   // workgroups before splitting
int64_t decode_batches(int64_t K);  // the smallest parts K is cut into
hipError_t launch_decode(const DecodeArgs& a, bool f32, Epi epi, hipStream_t s);

// A copy of an operand: out[rows][ld_out], columns zero-padded to ld_out (a
// multiple of 8); fp32 sources give three bf16 planes, out[3][rows][ld_out].
struct PackArgs {
  const void* src;
  uint16_t* out;
  int64_t rows, cols, ld, ld_out;
};
constexpr int kMaxPack = 6;
struct PackList {
  PackArgs t[kMaxPack];
  int32_t n, f32;
};
hipError_t launch_pack(const PackList& l, hipStream_t s);

enum NormKind { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

// Dropout factors of row `row`, columns [8 c, 8 c + 8): the half-words of
// Philox4x32-10 on the counter (c, row, row >> 32, offset) under the key
// `seed`; a half-word under `threshold` drops its element, the others are
// multiplied by `scale`. threshold = 0: no dropout.
struct DropArgs {
  uint32_t threshold, key0, key1, offset;
  float scale;
};

// r = alpha x + drop(gate * norm(z)), n = norm(r); z NULL: r = x. Element
// type f32 or bf16 for every array but the statistics.
struct NormArgs {
  const void *z, *x;
  void *r, *n;                       // r NULL with z NULL; n NULL with next_kind none
  const void *w_post, *b_post, *gate, *w_next, *b_next;  // NULL: 1, 0, 1, 1, 0
  float* stats;                      // [rows][4]: mean and 1 / deviation of z, of r
  // backward: upstream gradients dr (NULL: 0) and dn (NULL with next_kind
  // none), and the results (NULL: not wanted)
  const void *dr, *dn;
  void *dx, *dz;
  void *dw_post, *db_post, *dgate, *dw_next, *db_next;
  float* partial;                    // column sums, norm_partial_floats
  int64_t ldz, ldx, ldr, ldn, ld_gate, lddr, lddn, lddx, lddz, ld_dgate;
  int64_t rows, rows_per_gate;
  int32_t d, f32, post_kind, next_kind;
  float eps, alpha;
  DropArgs drop;
};
constexpr int kMaxNormWidth = 8192;
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s);
// What the rounding of bf16 n = norm(x) left, made again from x and the kept
// statistics (a.x, a.stats, a.w_next, a.b_next; a.n is read): out[rows][ld_out],
// columns zero-padded to ld_out (a multiple of 8).
hipError_t launch_norm_rest(const NormArgs& a, uint16_t* out, int64_t ld_out, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);
int64_t norm_partial_floats(const NormArgs& a);

struct DropoutArgs {
  const void* x;
  void* y;
  int64_t rows, cols, ldx, ldy;
  int32_t f32;
  DropArgs drop;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s);

}  // namespace shl
