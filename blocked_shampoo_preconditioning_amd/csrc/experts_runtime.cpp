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
                         a->ld_y, a->ld_xs, a->dweights};
  const hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const hipError_t err = what == kDispatch ? she::launch_dispatch(k, s) : what == kCombine ? she::launch_combine(k, s) : she::launch_combine_backward(k, s);
  return err == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(err, name);
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

}  // extern "C"
