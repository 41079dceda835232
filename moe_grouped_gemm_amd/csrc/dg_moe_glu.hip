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
// of the correctly rounded division. The reciprocal's result must not be below
// 2^-126, which it makes zero (from g = -87.4 on): a quarter of the sum is
// inverted, and a quarter of that taken. Below g = -88.7, where the exponential
// is infinite, the sigmoid is zero, as in the formula's float32 terms.
__device__ __forceinline__ float sigmoid(float g) {
  return 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(0.25f, __expf(-g), 0.25f));
}

// Rows of the no-padding layout that hold tokens: the counts' sum, negative
// counts as zero, cut at m. Computed by each wave for itself.
__device__ __forceinline__ int nopad_rows(const GluArgs& p) {
  long long n = 0;
  for (int g = threadIdx.x & 63; g < p.num_groups; g += 64) n += max(p.rows[g], 0);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  return (int)min(n, (long long)p.m);
}

// Row of the i-th turn of a group's workgroups, a permutation of each 8 << chunk
// rows: workgroups go round the 8 XCDs, and this gives an XCD 1 << chunk rows
// in succession, whose scales of a block are (part of) one line of sfa and fill it
// in one L2. Without it 32000 rows of 2048 wrote 79 MB where 66 are needed, and
// took a tenth more time. Which XCD comes first goes by the group: in the masked
// layout the first rows of every group hold tokens, the last ones none.
__device__ __forceinline__ int turn_row(int i, int g, int chunk) {
  const int low = (8 << chunk) - 1;
  return (i & ~low) + (((i + g) & 7) << chunk) + ((i & low) >> 3);
}

// Calls f(row of the buffer, group, row in the group, block) for every 128-value
// block of every row that holds a token, 16 lanes a block. A workgroup takes one
// row, or with MANY the `row_step` rows that 16 lanes a block leave it room for
// (an inner of at most 1024: 29416 rows of 256 take 9 us, a row a workgroup 26).
// With one row, whether it holds a token is the same in all lanes, asked before
// anything is stored, and so comes by scalar loads, soonest: with a loop over
// rows around it, 32000 rows of 2048 took a seventh more time. A row without a
// token costs its workgroup's launch: 16 us for 256 groups of 256 rows of 2048 of
// which 2 hold tokens (a fifth less with fewer workgroups that loop, but an eighth
// more with all rows held).
template <bool MANY, class F>
__device__ __forceinline__ void for_held_blocks(const GluArgs& p, int row_step, int chunk, F&& f) {
  const int blocks = p.inner / QBLOCK, at = threadIdx.x >> 4;
  const int g = blockIdx.y;
  int rows = p.m;  // rows below this hold tokens (contiguous: as their ids say)
  if (p.layout == DG_MOE_MASKED) rows = min(p.rows[g], p.m);
  if (p.layout == DG_MOE_NOPAD) rows = nopad_rows(p);
  if constexpr (MANY) {
    const int sub = at / blocks, r = blockIdx.x * row_step + sub;
    if (sub < row_step && r < rows && (p.layout != DG_MOE_CONTIGUOUS || p.rows[r] >= 0))
      f((size_t)g * p.m + r, g, r, at - sub * blocks);
  } else {
    const int r = turn_row(blockIdx.x, g, chunk);
    if (r < rows && (p.layout != DG_MOE_CONTIGUOUS || p.rows[r] >= 0))
      for (int b = at; b < blocks; b += blockDim.x >> 4) f((size_t)g * p.m + r, g, r, b);
  }
}

// Bound by memory: 4 bytes read and 1 + 4/128 written a value, about 20
// instructions each between. 32000 rows of 2048: 50 us (333 MB counted, 6.6 TB/s).
template <bool E8, bool MANY>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_fp8_kernel(GluArgs p, int row_step, int chunk) {
  const size_t I = p.inner;
  const int blocks = p.inner / QBLOCK, ld = align4(p.m), l16 = threadIdx.x & 15;
  for_held_blocks<MANY>(p, row_step, chunk, [&](size_t row, int g, int r, int b) {
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

// Bound by memory: 6 bytes read and 4 written a value. 29416 rows of 2048: 93 us
// (591 MB counted, 6.4 TB/s).
template <bool MANY>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_bwd_kernel(GluArgs p, int row_step, int chunk) {
  const size_t I = p.inner;
  const int l16 = threadIdx.x & 15;
  for_held_blocks<MANY>(p, row_step, chunk, [&](size_t row, int, int, int b) {
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

struct GluShape {
  dim3 grid;
  int threads, row_step, chunk;
};
GluShape glu_shape(const GluArgs& a) {
  const int pieces = a.inner / 8, groups = a.layout == DG_MOE_MASKED ? a.num_groups : 1;
  GluShape s{};
  s.row_step = std::max(1, 256 / pieces);
  if (s.row_step > 1) {
    s.threads = 256;
    s.grid = dim3((a.m + s.row_step - 1) / s.row_step, groups);
    return s;
  }
  s.threads = pass_threads(pieces, GLU_THREADS);
  for (s.chunk = 5; s.chunk > 0 && a.m < 8 << s.chunk;) --s.chunk;  // up to a line of sfa, 32 rows
  s.grid = dim3((a.m + (8 << s.chunk) - 1) / (8 << s.chunk) * (8 << s.chunk), groups);
  return s;
}

}  // namespace

hipError_t launch_swiglu_fp8(const GluArgs& a, bool ue8m0, hipStream_t stream) {
  const GluShape s = glu_shape(a);
  const bool many = s.row_step > 1;
  auto* kernel = ue8m0 ? (many ? swiglu_fp8_kernel<true, true> : swiglu_fp8_kernel<true, false>)
                       : (many ? swiglu_fp8_kernel<false, true> : swiglu_fp8_kernel<false, false>);
  hipLaunchKernelGGL(kernel, s.grid, dim3(s.threads), 0, stream, a, s.row_step, s.chunk);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const GluArgs& a, hipStream_t stream) {
  const GluShape s = glu_shape(a);
  auto* kernel = s.row_step > 1 ? swiglu_bwd_kernel<true> : swiglu_bwd_kernel<false>;
  hipLaunchKernelGGL(kernel, s.grid, dim3(s.threads), 0, stream, a, s.row_step, s.chunk);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
