// The gated activation between the two grouped GEMMs, quantised into the
// second one's FP8 operand, and its gradient.

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

constexpr int GLU_THREADS = 256;

// Rows of the no-padding layout that hold tokens: the counts' sum, negative
// counts as zero, cut at m. Computed by each wave for itself.
__device__ __forceinline__ int nopad_rows(const GluArgs& p) {
  long long n = 0;
  for (int g = threadIdx.x & 63; g < p.num_groups; g += 64) n += max(p.rows[g], 0);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  return (int)min(n, (long long)p.m);
}

// Does row r of group g hold a token?
__device__ __forceinline__ bool row_held(const GluArgs& p, int g, int r) {
  switch (p.layout) {
    case DG_MOE_CONTIGUOUS: return p.rows[r] >= 0;
    case DG_MOE_MASKED: return r < p.rows[g];
    case DG_MOE_NOPAD: return r < nopad_rows(p);
    default: return true;
  }
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// One workgroup a row; 16 lanes a 128-value block.
template <bool E8>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_fp8_kernel(GluArgs p) {
  const int r = blockIdx.x, g = blockIdx.y;
  if (!row_held(p, g, r)) return;
  const int blocks = p.inner / QBLOCK, ld = align4(p.m);
  const size_t row = (size_t)g * p.m + r, I = p.inner;
  for (int b = threadIdx.x >> 4; b < blocks; b += GLU_THREADS / 16) {
    const size_t c = (size_t)b * QBLOCK + (threadIdx.x & 15) * 8;
    const F8 gate = unpack8(load_stream16(p.gu + row * 2 * I + c)), up = unpack8(load_stream16(p.gu + row * 2 * I + I + c));
    F8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] = gate.v[i] * sigmoid(gate.v[i]) * up.v[i];
    float scale;
    store_stream(p.q + row * I + c, quantize_row<E8>(a, scale));
    if ((threadIdx.x & 15) == 0) p.sfa[((size_t)g * blocks + b) * ld + r] = scale;
  }
}

__global__ __launch_bounds__(GLU_THREADS) void swiglu_bwd_kernel(GluArgs p) {
  const int r = blockIdx.x, g = blockIdx.y;
  if (!row_held(p, g, r)) return;
  const size_t row = (size_t)g * p.m + r, I = p.inner;
  for (size_t c = threadIdx.x * 8; c < I; c += GLU_THREADS * 8) {
    const F8 gate = unpack8(load_stream16(p.gu + row * 2 * I + c)), up = unpack8(load_stream16(p.gu + row * 2 * I + I + c));
    const F8 da = unpack8(load_stream16(p.da + row * I + c));
    F8 dg, du;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(gate.v[i]), t = da.v[i] * s;
      dg.v[i] = t * up.v[i] * (1.0f + gate.v[i] * (1.0f - s));
      du.v[i] = t * gate.v[i];
    }
    store_stream(p.dgu + row * 2 * I + c, pack8(dg));
    store_stream(p.dgu + row * 2 * I + I + c, pack8(du));
  }
}

dim3 row_grid(const GluArgs& a) { return dim3(a.m, a.layout == DG_MOE_MASKED ? a.num_groups : 1); }

}  // namespace

hipError_t launch_swiglu_fp8(const GluArgs& a, bool ue8m0, hipStream_t stream) {
  hipLaunchKernelGGL(ue8m0 ? swiglu_fp8_kernel<true> : swiglu_fp8_kernel<false>, row_grid(a), dim3(GLU_THREADS), 0,
                     stream, a);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const GluArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(swiglu_bwd_kernel, row_grid(a), dim3(GLU_THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
