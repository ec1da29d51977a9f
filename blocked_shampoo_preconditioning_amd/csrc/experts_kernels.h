// Launchers of the experts' kernels (experts_route.hip), called by the host side
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
};
hipError_t launch_dispatch(const RouteArgs& a, hipStream_t s);
hipError_t launch_combine(const RouteArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const RouteArgs& a, hipStream_t s);

}  // namespace she
