// Internal interface between the C ABI of the steps around the GEMMs
// (dg_moe_api.cpp) and their kernels. Arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe/dg_moe.h"

namespace dg {
namespace moe {

constexpr int MAX_GROUPS = 4096;
constexpr int MAX_NOPAD = 2048;
constexpr int MAX_TOP_K = 32;
constexpr int SEGMENT = 128;     // row alignment of the contiguous layout
constexpr int QBLOCK = 128;      // values per scale
constexpr int MAX_NORM_HIDDEN = 16384;

inline __host__ __device__ int align4(int m) { return (m + 3) / 4 * 4; }

// Sorting and moving tokens (dg_moe_route.hip).
struct RouteArgs {
  int layout, tokens, top_k, num_groups, rows, hidden;
  const int32_t* ids;
  int32_t* row_of;
  int32_t* group_rows;
  int32_t* grouped_layout;
  void* workspace;
};
// Bytes of workspace that sorting up to `slots` slots takes.
long long sort_workspace(int slots, int num_groups);
hipError_t launch_sort(const RouteArgs& a, hipStream_t stream);
hipError_t launch_dispatch(const RouteArgs& a, const void* x, void* xp, hipStream_t stream);
hipError_t launch_dispatch_fp8(const RouteArgs& a, const void* x, void* q, float* sfa, bool ue8m0, hipStream_t stream);
hipError_t launch_combine(const RouteArgs& a, const void* yp, const float* w, void* y, hipStream_t stream);
hipError_t launch_combine_bwd(const RouteArgs& a, const void* dy, const void* yp, const float* w, void* dyp,
                              float* dw, hipStream_t stream);

// Gated activation (dg_moe_glu.hip).
struct GluArgs {
  const uint16_t* gu;
  const uint16_t* da;   // gradient only
  uint8_t* q;           // forward only
  float* sfa;           // forward only
  uint16_t* dgu;        // gradient only
  const int32_t* rows;
  int layout, m, num_groups, inner;
};
hipError_t launch_swiglu_fp8(const GluArgs& a, bool ue8m0, hipStream_t stream);
hipError_t launch_swiglu_bwd(const GluArgs& a, hipStream_t stream);

// Norms around the block (dg_moe_norm.hip).
// Most workgroups of the gradient's row loop (and rows of its partial sums).
int norm_bwd_grid(int tokens);
hipError_t launch_block_norm(const dg_moe_norm& a, int cus, hipStream_t stream);
hipError_t launch_block_norm_bwd(const dg_moe_norm_bwd& a, int cus, hipStream_t stream);

}  // namespace moe
}  // namespace dg
