// The gated activation between the two grouped GEMMs, quantised into the
// second one's FP8 or FP4 operand, and its gradient.

#include <algorithm>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

constexpr int GLU_THREADS = 512;  // at most

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
    if (l16 == 0) static_cast<float*>(p.sfa)[((size_t)g * blocks + b) * ld + r] = scale;
  });
}

// To FP4, one step of which is a quarter to a half of a value: the codes are those of
// the formula itself, whatever the last places of its float32 terms. With n = max(-g,
// 0) these are off by less than (1.5 n + 8) 2^-24: log2(e) g and its product round by 1.5
// |g| 2^-24 (no matter above zero, where the exponential is below 1 in a sum with 1), the
// exponential and the reciprocal by 2^-23 each, four operations by 2^-24. So a code or
// scale that comes out the same for values (n + 8) 2^-23 smaller and larger, n the
// block's largest, is the formula's. The others, a few values in 10^6, are computed again
// in 64 bits, a wave at a time, and so are blocks so small and gates so far below zero
// that float32 terms lose their precision.
constexpr uint32_t TINY = 0x0D800000u;  // 2^-100
constexpr float LOW_GATE = -87.0f;

__device__ __forceinline__ uint32_t swiglu_fp4_exact(u32x4 gate_raw, u32x4 up_raw, uint32_t* scale) {
  double a[8], top = 0.0;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double g = half_of(gate_raw[i / 2], i & 1), u = half_of(up_raw[i / 2], i & 1);
    a[i] = g / (1.0 + exp(-g)) * u;
    const double m = fabs(a[i]);
    finite &= m < 0x1.ffffffp127;  // what float32 rounds to infinity counts as that
    top = m > top ? m : top;
  }
  uint64_t bits = __builtin_bit_cast(uint64_t, top);
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const uint64_t other = __shfl_xor(bits, d);
    bits = bits > other ? bits : other;
  }
  uint32_t all = finite ? 1u : 0u;
  all = all & quad<0xB1>(all);
  all = all & quad<0x4E>(all);
  // As fp4_scale(), of a float64's exponent and mantissa (the exponent's offset is 1023).
  const int e = (int)((bits + 0x7FFFFFFFFFFFFull) >> 52) - (1023 - 127) - 2;
  const int code = bits == 0 ? 0 : max(e, 0);
  *scale = all ? (uint32_t)code : FP4_NAN_SCALE;
  if (!all) return 0;
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = ldexp(fabs(a[i]), 127 - code);
    const uint32_t c = (v > 0.25) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0);
    q |= (c | (signbit(a[i]) ? 8u : 0u)) << (4 * i);
  }
  return q;
}

__device__ __forceinline__ F8 scaled(const F8& a, float by) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = a.v[i] * by;
  return r;
}

// Bound by memory and the vector units about alike: 4 bytes read and 1/2 + 1/32
// written a value, and some 90 operations (exponential, reciprocal, two roundings to
// codes). 32000 rows of 2048: 57 us, 5.2 TB/s (295 MB); with a margin of 2^-17 for
// all gates, 6 times as many recomputed values, 61.
template <bool MANY>
__global__ __launch_bounds__(GLU_THREADS) void swiglu_fp4_kernel(GluArgs p, int row_step, int chunk) {
  const size_t I = p.inner;
  const int blocks = p.inner / QBLOCK, ld = align4(p.m), l16 = threadIdx.x & 15;
  for_held_blocks<MANY>(p, row_step, chunk, [&](size_t row, int g, int r, int b) {
    const uint16_t* src = p.gu + row * 2 * I + b * QBLOCK + l16 * 8;
    const u32x4 gate_raw = load_stream16(src), up_raw = load_stream16(src + I);
    const F8 gate = unpack8(gate_raw), up = unpack8(up_raw);
    F8 a;  // (with a sigmoid that is one operation short, and too small below LOW_GATE)
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] = gate.v[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-gate.v[i])) * up.v[i];
    const uint32_t top = max4(abs_top(a));
    uint32_t code = fp4_scale(top);
    float low = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) low = fminf(low, gate.v[i]);
    const float slack = __builtin_fmaf(__builtin_bit_cast(float, max4(abs_bits(low))), 0x1p-23f, 0x1p-20f);
    uint32_t q = fp4_codes(scaled(a, 1.0f - slack), code);
    const float amax = __builtin_bit_cast(float, top);
    bool near = q != fp4_codes(scaled(a, 1.0f + slack), code);
    near |= fp4_scale(abs_bits(amax * (1.0f - slack))) != fp4_scale(abs_bits(amax * (1.0f + slack)));
    if (__any(low < LOW_GATE || top < TINY)) {  // but a block of zeros is exact
      bool zero = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) zero &= gate.v[i] == 0.0f || up.v[i] == 0.0f;
      near |= (low < LOW_GATE || top < TINY) && !zero;
    }
    if (__any(near)) q = swiglu_fp4_exact(gate_raw, up_raw, &code);
    __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(p.q + (row * I + b * QBLOCK + l16 * 8) / 2));
    const uint32_t word = fp4_scale_word(code);
    if (l16 == 0) static_cast<uint32_t*>(p.sfa)[((size_t)g * blocks + b) * ld + r] = word;
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

hipError_t launch_swiglu_fp4(const GluArgs& a, hipStream_t stream) {
  const GluShape s = glu_shape(a);
  auto* kernel = s.row_step > 1 ? swiglu_fp4_kernel<true> : swiglu_fp4_kernel<false>;
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
