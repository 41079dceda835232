// The gated activation between the two grouped GEMMs, quantised into the
// second one's FP8 operand, and its gradient.

#include <algorithm>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

constexpr int GLU_THREADS = 512;  // at most

// 1 / (1 + exp(-g)) with the hardware's exponential and reciprocal, each good to
// an ulp or so (the exponential's argument rounds once, |g| 2^-24 more): far
// below the rounding of what is made of it, and a third of the instructions
// of the correctly rounded division.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// Rows of the no-padding layout that hold tokens: the counts' sum, negative
// counts as zero, cut at m. Computed by each wave for itself.
__device__ __forceinline__ int nopad_rows(const GluArgs& p) {
  long long n = 0;
  for (int g = threadIdx.x & 63; g < p.num_groups; g += 64) n += max(p.rows[g], 0);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  return (int)min(n, (long long)p.m);
}

// How workgroups share rows.
//   ROWS_ONE   one row a workgroup. Whether it holds a token is the same in all
//              lanes, asked before anything is stored, and so comes by scalar
//              loads, soonest: 57 us against 65 with a loop over rows around it
//              (32000 rows of 2048, contiguous layout).
//   ROWS_LOOP  as many workgroups as fill the device a few times, each going on
//              to later rows of its group: for the masked layout where G * max_m
//              rows, most of them empty in decoding, would each cost a workgroup:
//              2 rows in each of 256 groups of 256 take 10.4 us, a row a
//              workgroup 16.8 (and full groups 114 against 109).
//   ROWS_MANY  several rows a workgroup, 16 lanes a block, for an inner of at
//              most 1024: 29416 rows of 256 take 10 us, a row a workgroup 25.
enum { ROWS_ONE, ROWS_LOOP, ROWS_MANY };

// Calls f(row of the buffer, group, row in the group, block) for every 128-value
// block of every row that holds a token.
template <int MODE, class F>
__device__ __forceinline__ void for_held_blocks(const GluArgs& p, int row_step, F&& f) {
  const int blocks = p.inner / QBLOCK, at = threadIdx.x >> 4;
  const int g = blockIdx.y;
  int rows = p.m;  // rows below this hold tokens (contiguous: as their ids say)
  if (p.layout == DG_MOE_MASKED) rows = min(p.rows[g], p.m);
  if (p.layout == DG_MOE_NOPAD) rows = nopad_rows(p);
  auto row_blocks = [&](int r) {
    for (int b = at; b < blocks; b += blockDim.x >> 4) f((size_t)g * p.m + r, g, r, b);
  };
  if constexpr (MODE == ROWS_ONE) {
    const int r = blockIdx.x;
    if (r < rows && (p.layout != DG_MOE_CONTIGUOUS || p.rows[r] >= 0)) row_blocks(r);
  } else if constexpr (MODE == ROWS_LOOP) {
    for (int r = blockIdx.x; r < rows; r += gridDim.x) row_blocks(r);
  } else {
    const int sub = at / blocks, b = at - sub * blocks;
    if (sub >= row_step) return;
    for (int r = blockIdx.x * row_step + sub; r < rows; r += gridDim.x * row_step)
      if (p.layout != DG_MOE_CONTIGUOUS || p.rows[r] >= 0) f((size_t)g * p.m + r, g, r, b);
  }
}

// Bound by memory: 4 bytes read and 1 + 4/128 written a value, about 20
// instructions each between.
template <bool E8, int MODE>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_fp8_kernel(GluArgs p, int row_step) {
  const size_t I = p.inner;
  const int blocks = p.inner / QBLOCK, ld = align4(p.m), l16 = threadIdx.x & 15;
  for_held_blocks<MODE>(p, row_step, [&](size_t row, int g, int r, int b) {
    const uint16_t* src = p.gu + row * 2 * I + b * QBLOCK + l16 * 8;
    const u32x4 gate_raw = load_stream16(src), up_raw = load_stream16(src + I);
    const F8 gate = unpack8(gate_raw), up = unpack8(up_raw);
    F8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] = gate.v[i] * sigmoid(gate.v[i]) * up.v[i];
    float scale;
    store_stream(p.q + row * I + b * QBLOCK + l16 * 8, quantize_row<E8>(a, scale));
    if (l16 == 0) p.sfa[((size_t)g * blocks + b) * ld + r] = scale;
  });
}

// Bound by memory: 6 bytes read and 4 written a value.
template <int MODE>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_bwd_kernel(GluArgs p, int row_step) {
  const size_t I = p.inner;
  const int l16 = threadIdx.x & 15;
  for_held_blocks<MODE>(p, row_step, [&](size_t row, int, int, int b) {
    const size_t c = b * QBLOCK + l16 * 8;
    const u32x4 gate_raw = load_stream16(p.gu + row * 2 * I + c), up_raw = load_stream16(p.gu + row * 2 * I + I + c);
    const u32x4 da_raw = load_stream16(p.da + row * I + c);
    const F8 gate = unpack8(gate_raw), up = unpack8(up_raw), da = unpack8(da_raw);
    F8 dg, du;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(gate.v[i]), t = da.v[i] * s;
      dg.v[i] = t * up.v[i] * (1.0f + gate.v[i] * (1.0f - s));
      du.v[i] = t * gate.v[i];
    }
    store_stream(p.dgu + row * 2 * I + c, pack8(dg));
    store_stream(p.dgu + row * 2 * I + I + c, pack8(du));
  });
}

// Most workgroups of the masked layout.
constexpr int MASKED_WORKGROUPS = 16384;

struct GluShape {
  dim3 grid;
  int threads, row_step, mode;
};
GluShape glu_shape(const GluArgs& a) {
  const int pieces = a.inner / 8;
  GluShape s;
  s.row_step = std::max(1, 256 / pieces);
  s.mode = s.row_step > 1 ? ROWS_MANY : ROWS_ONE;
  s.threads = s.row_step > 1 ? 256 : even_threads(pieces, GLU_THREADS);
  const int steps = (a.m + s.row_step - 1) / s.row_step;
  s.grid = dim3(steps);
  if (a.layout == DG_MOE_MASKED) {
    const int most = std::max(1, MASKED_WORKGROUPS / a.num_groups);
    if (steps > most && s.mode == ROWS_ONE) s.mode = ROWS_LOOP;
    s.grid = dim3(std::min(steps, most), a.num_groups);
  }
  return s;
}

template <int MODE>
void launch_fp8(const GluArgs& a, const GluShape& s, bool ue8m0, hipStream_t stream) {
  hipLaunchKernelGGL((ue8m0 ? swiglu_fp8_kernel<true, MODE> : swiglu_fp8_kernel<false, MODE>), s.grid, dim3(s.threads),
                     0, stream, a, s.row_step);
}

}  // namespace

hipError_t launch_swiglu_fp8(const GluArgs& a, bool ue8m0, hipStream_t stream) {
  const GluShape s = glu_shape(a);
  if (s.mode == ROWS_ONE) launch_fp8<ROWS_ONE>(a, s, ue8m0, stream);
  else if (s.mode == ROWS_LOOP) launch_fp8<ROWS_LOOP>(a, s, ue8m0, stream);
  else launch_fp8<ROWS_MANY>(a, s, ue8m0, stream);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const GluArgs& a, hipStream_t stream) {
  const GluShape s = glu_shape(a);
  auto* kernel = s.mode == ROWS_ONE    ? swiglu_bwd_kernel<ROWS_ONE>
                 : s.mode == ROWS_LOOP ? swiglu_bwd_kernel<ROWS_LOOP>
                                       : swiglu_bwd_kernel<ROWS_MANY>;
  hipLaunchKernelGGL(kernel, s.grid, dim3(s.threads), 0, stream, a, s.row_step);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
