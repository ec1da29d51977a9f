// Host side of include/shampoo_experts.h: argument checks, the workspaces'
// layout and the launches of the experts' path.
#include "../../include/shampoo_experts.h"

#include <exception>

#include "experts_kernels.h"
#include "runtime_common.h"

using shp_rt::fail;

namespace {

constexpr int64_t kMaxTotal = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxWidth = int64_t(1) << 21;
constexpr int64_t kAnyLd = int64_t(1) << 40;

bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

#define RC(expr)                  \
  do {                            \
    if (int rc_ = (expr)) return rc_; \
  } while (0)

// No C++ exception crosses the C boundary.
template <class F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(SHAMPOO_ERR_INVALID_ARG, e.what());
  } catch (...) {
    return fail(SHAMPOO_ERR_INVALID_ARG, "unknown C++ exception");
  }
}

int invalid(const std::string& msg) { return fail(SHAMPOO_ERR_INVALID_ARG, msg); }

// A matrix or, with ld = cols, an array; nothing is asked of an empty one.
int check_array(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize, int64_t max_ld = kAnyLd) {
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (!p) return invalid(std::string(name) + " is NULL");
  if (ld < cols || ld > max_ld)
    return invalid(std::string(name) + ": leading dimension " + std::to_string(ld) + " is not in [" + std::to_string(cols) + ", " +
                   std::to_string(max_ld) + "]");
  if (!aligned(p, esize)) return fail(SHAMPOO_ERR_MISALIGNED, std::string(name) + " is not aligned to its element size");
  return SHAMPOO_OK;
}

int check_dtype(int32_t dtype) {
  if (dtype != SHAMPOO_F32 && dtype != SHAMPOO_BF16)
    return fail(SHAMPOO_ERR_UNSUPPORTED, "dtype must be SHAMPOO_F32 or SHAMPOO_BF16");
  return SHAMPOO_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SHAMPOO_OK;
  if (!ws) return invalid("workspace is NULL");
  if (!aligned(ws, 256)) return fail(SHAMPOO_ERR_MISALIGNED, "workspace is not aligned to 256 bytes");
  if (have < need)
    return fail(SHAMPOO_ERR_WORKSPACE_TOO_SMALL,
                "workspace has " + std::to_string(have) + " bytes, the call needs " + std::to_string(need));
  return SHAMPOO_OK;
}

int check_counts(int64_t tokens, int64_t slots) {
  if (slots < 1 || slots > 1024) return invalid("slots must be in [1, 1024]");
  if (tokens < 0 || tokens > kMaxTotal / slots) return invalid("tokens must be at least 0 and tokens * slots at most 2^31 - 1024");
  return SHAMPOO_OK;
}

// -------------------------------------------------------- tokens by expert
int check_sort(const shampoo_sort_t* a) {
  if (!a) return invalid("arguments are NULL");
  RC(check_counts(a->tokens, a->slots));
  if (a->experts < 1 || a->experts > 1024) return invalid("experts must be in [1, 1024]");
  if (a->id_bytes != 4 && a->id_bytes != 8) return fail(SHAMPOO_ERR_UNSUPPORTED, "id_bytes must be 4 or 8");
  return SHAMPOO_OK;
}

size_t sort_workspace(const shampoo_sort_t* a) {
  uint32_t blocks, per_block;
  she::sort_plan(a->tokens * a->slots, blocks, per_block);
  return blocks > 1 ? size_t(4) * blocks * (a->experts + 1) : 0;
}

enum Route { kDispatch, kCombine, kCombineBackward };

int route(const shampoo_route_t* a, Route what, const char* name, void* hip_stream) {
  if (!a) return invalid("arguments are NULL");
  RC(check_counts(a->tokens, a->slots));
  if (a->width < 0 || a->width > kMaxWidth) return invalid("width must be in [0, 2^21]");
  RC(check_dtype(a->dtype));
  const int64_t e = a->dtype == SHAMPOO_F32 ? 4 : 2, total = a->tokens * a->slots;
  RC(check_array("rows", a->rows, a->tokens, a->slots, a->slots, 4));
  if (a->weights && what != kDispatch) RC(check_array("weights", a->weights, a->tokens, a->slots, a->slots, 4));
  if (what == kDispatch || what == kCombineBackward) {
    RC(check_array(what == kDispatch ? "x" : "dy", a->x, a->tokens, a->width, a->ld_x, e));
    RC(check_array(what == kDispatch ? "xs" : "dys", a->xs, total, a->width, a->ld_xs, e));
  }
  if (what != kDispatch) RC(check_array("ys", a->ys, total, a->width, a->ld_ys, e));
  if (what == kCombine) RC(check_array("y", a->y, a->tokens, a->width, a->ld_y, e));
  if (what == kCombineBackward) {
    RC(check_array("dweights", a->dweights, a->tokens, a->slots, a->slots, 4));
    if (total > 0 && !a->weights) return invalid("weights is NULL: without weights the gradient is a dispatch of dy");
  }
  const she::RouteArgs k{a->tokens, static_cast<uint32_t>(a->slots), static_cast<uint32_t>(total), static_cast<int32_t>(a->width),
                         a->dtype == SHAMPOO_F32 ? 1 : 0, a->rows, a->weights, a->x, a->ys, a->ld_x, a->ld_ys, a->y, a->xs,
                         a->ld_y, a->ld_xs, a->dweights, aligned(a->xs, 128) && a->ld_xs * e % 128 == 0};
  const hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const hipError_t err = what == kDispatch ? she::launch_dispatch(k, s) : what == kCombine ? she::launch_combine(k, s) : she::launch_combine_backward(k, s);
  return err == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(err, name);
}

// -------------------------------------------------------- products in 8 bits
constexpr int64_t kMaxRows = (int64_t(1) << 31) - (int64_t(1) << 18);  // padded rows of 1024 experts stay in 32 bits

constexpr int64_t kMaxSavedRows = (int64_t(1) << 23) - (int64_t(1) << 18);  // 256 columns of them stay within 32-bit byte offsets

int64_t blocks_of(int64_t n) { return (n + she::kBlock - 1) / she::kBlock; }

int check_sizes(int64_t in, int64_t out, int32_t experts, int32_t dtype) {
  if (in < 1 || in > kMaxWidth || out < 1 || out > kMaxWidth) return invalid("in and out must be in [1, 2^21]");
  if (experts < 1 || experts > 1024) return invalid("experts must be in [1, 1024]");
  return check_dtype(dtype);
}

int check_aligned(const char* name, const void* p, int64_t a) {
  if (!p) return invalid(std::string(name) + " is NULL");
  if (!aligned(p, a)) return fail(SHAMPOO_ERR_MISALIGNED, std::string(name) + " is not aligned to " + std::to_string(a) + " bytes");
  return SHAMPOO_OK;
}

// Matrices one behind the other, or side by side in rows that hold a row of each.
int check_matrices(const char* name, const void* p, int64_t experts, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int64_t esize) {
  RC(check_array(name, p, rows, cols, ld, esize));
  if (experts == 1) return SHAMPOO_OK;
  const bool behind = stride >= (rows - 1) * ld + cols && stride <= kAnyLd;
  const bool beside = stride >= cols && stride <= ld && (experts - 1) * stride + cols <= ld;
  if (!behind && !beside) return invalid(std::string(name) + ": matrices overlap, or lie over 2^40 elements apart");
  return SHAMPOO_OK;
}

int check_product(const shampoo_product8_t* a) {
  if (!a) return invalid("arguments are NULL");
  if (a->rows < 0 || a->rows > kMaxRows) return invalid("rows must be in [0, 2^31 - 2^18]");
  RC(check_sizes(a->in, a->out, a->experts, a->dtype));
  if (!a->offsets && a->experts > 1) return invalid("offsets is NULL: with several experts it says which rows are whose");
  if (a->offsets) RC(check_aligned("offsets", a->offsets, 4));
  if (a->source) {
    if (!a->offsets) return invalid("source is given without offsets");
    RC(check_aligned("source", a->source, 4));
    if (a->slots < 1 || a->slots > 1024) return invalid("slots must be in [1, 1024]");
    if (a->x_rows < (a->rows > 0 ? 1 : 0) || a->x_rows > kMaxTotal) return invalid("x_rows must be in [1, 2^31 - 1024]");
    if (a->slot_rows) {
      RC(check_aligned("slot_rows", a->slot_rows, 4));
      if (a->rows != a->x_rows * a->slots) return invalid("rows must be x_rows * slots with slot_rows");
    }
  }
  return SHAMPOO_OK;
}

// Blocks of 128 padded rows that all experts' rows can take.
int64_t row_blocks(const shampoo_product8_t* a) {
  if (!a->offsets) return blocks_of(a->rows);
  const int64_t e = a->experts < a->rows ? a->experts : a->rows;
  return (a->rows + (she::kBlock - 1) * e) / she::kBlock;
}

// The tile of a launch's products, by an estimate of its time in microseconds. A K
// block takes a 256 tile alone on its CU 1.5, each of two 128 tiles on one 1.0; a tile
// costs 2 besides, the launch 5. 256 tiles go in whole rounds over the CUs, while
// 128 tiles that are left alone on a CU go faster. Of an expert's rows the last tile
// is half empty in the mean. Measured, both sides in turn on one card, median launch, 256
// and 128, us: y of 8192 x 2048 x 8192 127 and 145, dx and dW of it 219 and 264; of
// 4096 x 8192 x 2048 84 and 64, 118 and 143; of 16384 rows of 64 experts x 2048 x 768
// 63 and 41, 133 and 142, of eight x 2048 x 2048 81 and 76, 152 and 164; of 1024 x 768 x
// 2048 15 and 9, 25 and 14.
// Where 128 tiles of bf16 are no more than CUs, four steps of each are on their way: for
// long sums (four and two, y of 512 x 8192 x 512 34 and 41, of 256 x 2048 x 8192 14.5 and
// 17.6; dx and dW of 1024 x 768 x 2048 13.6 and 14.2); short ones lose up to 0.7 (y of
// 1024 x 512 x 1024 7.3 and 6.6). fp32 has no such tile, it was slower for long sums too
// (512 x 8192 x 512 62 and 54, 1024 x 768 x 2048 13.9 and 12.4).
she::ProductTile choose_tile(const shampoo_product8_t* a, bool backward) {
  const bool dx = !backward || a->dx, dw = backward && a->dw;
  const double experts = a->experts, rows = static_cast<double>(a->rows);
  auto estimate = [&](int64_t side, double step, double slots, double& tiles) {
    auto across = [&](int64_t n) { return static_cast<double>((n + side - 1) / side); };
    const double used = a->offsets ? experts < rows ? experts : rows : 0;
    const double n = dx ? (a->offsets ? rows / static_cast<double>(side) + used / 2 : across(a->rows)) * across(backward ? a->in : a->out) : 0;
    const double c = dw ? across(a->in) * across(a->out) * experts : 0;
    const double row_steps = static_cast<double>(blocks_of(backward ? a->out : a->in)), col_steps = rows / 128 / experts + 0.5;
    tiles = n + c;
    double rounds = tiles / slots;
    if (side == 256) rounds = static_cast<double>(static_cast<int64_t>(rounds + 0.999));
    if (rounds < 1) rounds = 1;
    return tiles > 0 ? rounds * ((n * row_steps + c * col_steps) / tiles * step + 2) : 0;
  };
  double large, small;
  const double us_large = estimate(256, 1.5, 256, large), us_small = estimate(128, 1.0, 512, small);
  if (a->dtype != SHAMPOO_F32 && us_large < us_small) return she::kProduct256;
  return a->dtype != SHAMPOO_F32 && small <= 256 ? she::kProduct128Deep : she::kProduct128;
}

// Quantized operands by rows and by columns in the workspace, and the products of a
// call with their work, also in the workspace.
struct ProductPlan {
  int64_t blocks = 0;
  shp_rt::Carver ws;
  she::QuantizeArgs q{};
};

size_t saved_size(const shampoo_product8_t* a) {
  shp_rt::Carver c;
  const int64_t nb = row_blocks(a), ib = blocks_of(a->in);
  if (nb == 0) return 0;
  c.take(nb * ib * she::kBlock * she::kBlock);
  c.take(nb * ib * she::kBlock);
  return static_cast<size_t>(c.o);
}

// Up to 64 rows that nothing is kept of go in one launch without a workspace. The host
// knows how many rows there are, not whose. Measured, in one launch and in two with 128
// tiles, us a call (calls in a graph, weights from memory), bf16: 2048 x 8192 1 row 8
// and 18, 16 rows 8 and 19, 32 14 and 19, 48 19 and 19, 64 24 and 19; 512 x 1024 64 rows 8
// and 10; 2048 x 2048 48 14 and 17, 64 18 and 17; eight experts of 2048 x 8192 64 rows
// 35 and 36, 96 43 and 36; 64 experts of 2048 x 768, 8 a token, 64 24 and 26, 512 29 and
// 37; 64 of 2048 x 2048, 2 a token, 48 40 and 47, 64 53 and 49, 128 58 and 58; 16 of 512 x
// 1024 64 9 and 13. fp32: 2048 x 8192 48 24 and 27, 64 30 and 27; eight experts 64 35 and
// 41. One matrix of more columns or K is the exception: 33 rows of 8192 x 8192 57 and 45, of
// 2048 x 16384 35 and 19.
bool few_rows(const shampoo_product8_t* a, bool backward) {
  return a->rows <= she::kFewRows && !(backward ? a->dw : a->saved);
}

// y or dx: rows of tokens, quantized by rows, against the weights.
she::ProductArgs row_product(const shampoo_product8_t* a, int64_t blocks, const void* values, const void* scales, int64_t k, int64_t n, void* c,
                             int64_t ldc) {
  const int64_t kb = blocks_of(k), nb = blocks_of(n), scale_pitch = (kb + 3) / 4 * 4;
  she::ProductArgs g{};
  g.b = static_cast<const uint8_t*>(values);
  g.b_scales = static_cast<const uint8_t*>(scales);
  g.pitch = kb * she::kBlock;
  g.size_a = blocks * she::kBlock * g.pitch;
  g.size_b = g.b_stride = n * g.pitch;
  g.b_scale_stride = nb * scale_pitch;
  g.a_blocks = static_cast<int32_t>(blocks);
  g.b_blocks = static_cast<int32_t>(nb);
  g.b_scale_pitch = static_cast<int32_t>(scale_pitch);
  g.M = static_cast<int32_t>(a->rows);
  g.N = static_cast<int32_t>(n);
  g.k_blocks = static_cast<int32_t>(kb);
  g.c = c;
  g.ldc = ldc;
  return g;
}

// dW: what was saved of x against dy, both by columns.
she::ProductArgs column_product(const shampoo_product8_t* a, int64_t blocks) {
  const int64_t ib = blocks_of(a->in), ob = blocks_of(a->out);
  she::ProductArgs g{};
  g.pitch = blocks * she::kBlock;
  g.a = static_cast<const uint8_t*>(a->saved);
  g.a_scales = g.a + shp_rt::align_up(ib * she::kBlock * g.pitch);
  g.size_a = ib * she::kBlock * g.pitch;
  g.size_b = ob * she::kBlock * g.pitch;
  g.a_blocks = static_cast<int32_t>(ib);
  g.b_blocks = static_cast<int32_t>(ob);
  g.M = static_cast<int32_t>(a->in);
  g.N = static_cast<int32_t>(a->out);
  g.k_blocks = static_cast<int32_t>(blocks);
  g.by_expert = 1;
  g.c = a->dw;
  g.ldc = a->ld_dw;
  g.c_stride = a->stride_dw;
  return g;
}

// A call's quantization and products, at `ws`; sizes are the same wherever that is.
ProductPlan plan_product(const shampoo_product8_t* a, bool backward, void* ws) {
  ProductPlan p;
  p.blocks = row_blocks(a);
  const bool dw = backward && a->dw;
  if (few_rows(a, backward) || (p.blocks == 0 && !dw)) return p;
  const int64_t k = backward ? a->out : a->in, kb = blocks_of(k), bytes = p.blocks * kb * she::kBlock * she::kBlock;
  auto take = [&](int64_t n) { return static_cast<uint8_t*>(ws) + p.ws.take(n); };
  she::QuantizeArgs& q = p.q;
  q.x = backward ? a->dy : a->x;
  q.ld = backward ? a->ld_dy : a->ld_x;
  q.f32 = a->dtype == SHAMPOO_F32;
  q.cols = static_cast<int32_t>(k);
  q.col_blocks = static_cast<int32_t>(kb);
  q.g = she::Groups{a->offsets, static_cast<int32_t>(a->rows), a->experts, static_cast<int32_t>(p.blocks)};
  const bool gather = !backward && a->source;
  q.source = gather ? a->source : nullptr;
  q.slots = static_cast<uint32_t>(gather ? a->slots : 1);
  q.rows_in = static_cast<int32_t>(gather ? a->x_rows : a->rows);
  if (gather && !a->saved && a->slot_rows && a->slots >= 2 && a->slots <= she::kMaxScatter) q.slot_rows = a->slot_rows;
  she::Products& g = q.products;
  g.experts = a->experts;
  g.f32 = q.f32;
  g.tile = choose_tile(a, backward);
  if (p.blocks > 0 && (!backward || a->dx)) {
    q.by_rows = take(bytes);
    q.row_scales = take(bytes / she::kBlock);
    she::ProductArgs& r = g.p[g.count++];
    r = backward ? row_product(a, p.blocks, a->back_values, a->back_scales, a->out, a->in, a->dx, a->ld_dx)
                 : row_product(a, p.blocks, a->values, a->scales, a->in, a->out, a->y, a->ld_y);
    r.a = q.by_rows;
    r.a_scales = q.row_scales;
  }
  if (dw) {
    q.by_cols = take(bytes);
    q.col_scales = take(bytes / she::kBlock);
    she::ProductArgs& c = g.p[g.count++];
    c = column_product(a, p.blocks);
    c.b = q.by_cols;
    c.b_scales = q.col_scales;
  } else if (!backward && a->saved) {
    q.by_cols = static_cast<uint8_t*>(a->saved);
    q.col_scales = q.by_cols + shp_rt::align_up(bytes);
  }
  const int64_t per = she::work_length(g, a->rows, a->offsets != nullptr);
  g.per = static_cast<int32_t>(per);
  g.work = reinterpret_cast<she::WorkRecord*>(take(8 * per * static_cast<int64_t>(sizeof(she::WorkRecord))));
  return p;
}

hipError_t run_products(const ProductPlan& p, hipStream_t s) {
  const hipError_t e = she::launch_quantize(p.q, s);
  return e == hipSuccess && p.q.products.count ? she::launch_products(p.q.products, s) : e;
}

hipError_t few_product(const shampoo_product8_t* a, bool gather, const void* x, int64_t ld, const void* values, const void* scales, int64_t k, int64_t n,
                       void* c, int64_t ldc, hipStream_t s) {
  const int64_t kb = blocks_of(k), scale_pitch = (kb + 3) / 4 * 4;
  she::FewArgs f{};
  f.x = x;
  f.ld_x = ld;
  f.g = she::Groups{a->offsets, static_cast<int32_t>(a->rows), a->experts, 0};
  f.slots = 1;
  f.rows_in = static_cast<int32_t>(a->rows);
  f.b = static_cast<const uint8_t*>(values);
  f.b_scales = static_cast<const uint8_t*>(scales);
  f.pitch_b = kb * she::kBlock;
  f.b_stride = n * f.pitch_b;
  f.b_scale_stride = blocks_of(n) * scale_pitch;
  f.b_scale_pitch = static_cast<int32_t>(scale_pitch);
  f.K = static_cast<int32_t>(k);
  f.N = static_cast<int32_t>(n);
  f.c = c;
  f.ldc = ldc;
  f.f32 = a->dtype == SHAMPOO_F32;
  if (gather) {
    f.source = a->source;
    f.slots = static_cast<uint32_t>(a->slots);
    f.rows_in = static_cast<int32_t>(a->x_rows);
  }
  return she::launch_few(f, s);
}

int forward(const shampoo_product8_t* a, void* ws, size_t ws_bytes, hipStream_t s) {
  const int64_t esize = a->dtype == SHAMPOO_F32 ? 4 : 2;
  RC(check_aligned("values", a->values, 16));
  RC(check_aligned("scales", a->scales, 4));
  RC(check_array("x", a->x, a->source ? a->x_rows : a->rows, a->in, a->ld_x, esize));
  RC(check_array("y", a->y, a->rows, a->out, a->ld_y, esize));
  if (a->saved && !aligned(a->saved, 256)) return fail(SHAMPOO_ERR_MISALIGNED, "saved is not aligned to 256 bytes");
  if (a->saved && a->rows > kMaxSavedRows) return invalid("rows must be at most 2^23 - 2^18 where they are saved for dw");
  const ProductPlan p = plan_product(a, false, ws);
  RC(check_workspace(ws, ws_bytes, static_cast<size_t>(p.ws.o)));
  if (a->rows == 0) return SHAMPOO_OK;
  const hipError_t e = few_rows(a, false)
                           ? few_product(a, a->source != nullptr, a->x, a->ld_x, a->values, a->scales, a->in, a->out, a->y, a->ld_y, s)
                           : run_products(p, s);
  return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_product8_forward");
}

int backward(const shampoo_product8_t* a, void* ws, size_t ws_bytes, hipStream_t s) {
  const int64_t esize = a->dtype == SHAMPOO_F32 ? 4 : 2;
  if (!a->dx && !a->dw) return SHAMPOO_OK;
  RC(check_array("dy", a->dy, a->rows, a->out, a->ld_dy, esize));
  if (a->dx) {
    RC(check_aligned("back_values", a->back_values, 16));
    RC(check_aligned("back_scales", a->back_scales, 4));
    RC(check_array("dx", a->dx, a->rows, a->in, a->ld_dx, esize));
  }
  if (a->dw) {
    if (a->rows > kMaxSavedRows) return invalid("rows must be at most 2^23 - 2^18 where dw is wanted");
    if (a->rows > 0) RC(check_aligned("saved", a->saved, 256));
    RC(check_matrices("dw", a->dw, a->experts, a->in, a->out, a->ld_dw, a->stride_dw, esize));
  }
  const ProductPlan p = plan_product(a, true, ws);
  RC(check_workspace(ws, ws_bytes, static_cast<size_t>(p.ws.o)));
  if (a->rows == 0 && !a->dw) return SHAMPOO_OK;
  const hipError_t e = few_rows(a, true)
                           ? few_product(a, false, a->dy, a->ld_dy, a->back_values, a->back_scales, a->out, a->in, a->dx, a->ld_dx, s)
                           : run_products(p, s);
  return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_product8_backward");
}

}  // namespace

extern "C" {

int shampoo_sort_workspace_size(const shampoo_sort_t* a, size_t* bytes_out) {
  return guarded([&]() -> int {
    RC(check_sort(a));
    if (!bytes_out) return invalid("bytes_out is NULL");
    *bytes_out = sort_workspace(a);
    return SHAMPOO_OK;
  });
}

int shampoo_sort_tokens(const shampoo_sort_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_sort(a));
    RC(check_array("ids", a->ids, a->tokens, a->slots, a->ld_ids, a->id_bytes));
    RC(check_array("offsets", a->offsets, 1, a->experts + 1, a->experts + 1, 4));
    RC(check_array("rows", a->rows, a->tokens, a->slots, a->slots, 4));
    RC(check_array("source", a->source, a->tokens, a->slots, a->slots, 4));
    RC(check_workspace(workspace, workspace_bytes, sort_workspace(a)));
    she::SortArgs k{a->ids, a->ld_ids, static_cast<uint32_t>(a->slots), static_cast<uint32_t>(a->tokens * a->slots),
                    static_cast<uint32_t>(a->experts), 0, 0, a->id_bytes == 8 ? 1 : 0, a->offsets, a->rows, a->source,
                    static_cast<uint32_t*>(workspace)};
    she::sort_plan(k.total, k.blocks, k.per_block);
    const hipError_t e = she::launch_sort(k, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_sort_tokens");
  });
}

int shampoo_dispatch(const shampoo_route_t* a, void* hip_stream) {
  return guarded([&] { return route(a, kDispatch, "shampoo_dispatch", hip_stream); });
}

int shampoo_combine(const shampoo_route_t* a, void* hip_stream) {
  return guarded([&] { return route(a, kCombine, "shampoo_combine", hip_stream); });
}

int shampoo_combine_backward(const shampoo_route_t* a, void* hip_stream) {
  return guarded([&] { return route(a, kCombineBackward, "shampoo_combine_backward", hip_stream); });
}

int shampoo_quantize_weight(const shampoo_weight8_t* a, void* hip_stream) {
  return guarded([&]() -> int {
    if (!a) return invalid("arguments are NULL");
    RC(check_sizes(a->in, a->out, a->experts, a->dtype));
    RC(check_matrices("w", a->w, a->experts, a->in, a->out, a->ld_w, a->stride_w, a->dtype == SHAMPOO_F32 ? 4 : 2));
    RC(check_aligned("values", a->values, 16));
    RC(check_aligned("scales", a->scales, 4));
    if (a->back_values || a->back_scales) {
      RC(check_aligned("back_values", a->back_values, 16));
      RC(check_aligned("back_scales", a->back_scales, 4));
    }
    const she::WeightArgs k{a->w, a->ld_w, a->stride_w, a->dtype == SHAMPOO_F32 ? 1 : 0, a->experts, static_cast<int32_t>(a->in),
                            static_cast<int32_t>(a->out), static_cast<uint8_t*>(a->values), static_cast<uint8_t*>(a->scales),
                            static_cast<uint8_t*>(a->back_values), static_cast<uint8_t*>(a->back_scales)};
    const hipError_t e = she::launch_quantize_weight(k, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_quantize_weight");
  });
}

int shampoo_product8_saved_size(const shampoo_product8_t* a, size_t* bytes_out) {
  return guarded([&]() -> int {
    RC(check_product(a));
    if (!bytes_out) return invalid("bytes_out is NULL");
    *bytes_out = saved_size(a);
    return SHAMPOO_OK;
  });
}

int shampoo_product8_workspace_size(const shampoo_product8_t* a, int32_t backward, size_t* bytes_out) {
  return guarded([&]() -> int {
    RC(check_product(a));
    if (!bytes_out) return invalid("bytes_out is NULL");
    *bytes_out = static_cast<size_t>(plan_product(a, backward != 0, nullptr).ws.o);
    return SHAMPOO_OK;
  });
}

int shampoo_product8_forward(const shampoo_product8_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_product(a));
    return forward(a, workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
  });
}

int shampoo_product8_backward(const shampoo_product8_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_product(a));
    return backward(a, workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
  });
}

}  // extern "C"
