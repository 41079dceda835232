// Device code shared by the steps around the GEMMs: BF16 vectors, sums over
// a wave, and the quantisation of a 128-value block.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "dg_moe_internal.h"

namespace dg {
namespace moe {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int I, int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

struct F8 {
  float v[8];
};

__device__ __forceinline__ u32x4 load16(const void* p) { return *reinterpret_cast<const u32x4*>(p); }

// Streaming (non-temporal) accesses: the line is not kept in L2 for its own
// sake. For rows that a kernel reads or writes once. Time with plain ones over
// time with streaming ones, at the largest sizes: combine of 65536 rows of 7168
// 1.15, its gradient with the dispatch's 1.07, the activation 1.13 and its
// gradient 1.11, the norms 1.06, their gradient 1.10, FP8 dispatch 1.11, BF16
// dispatch 1.06 (whose tokens are read by plain loads: streaming ones 1.05). The
// next call that reads such a row loses nothing: a whole block (dispatch,
// product, activation, product, combine, norm; 16 experts, rows of 7168 and
// 2048) takes 1.00 of the time with plain ones for 5 tokens, 0.98 for 64 and 256
// and 1.00 for 1024 and 4096.
__device__ __forceinline__ u32x4 load_stream16(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
template <class T>
__device__ __forceinline__ void store_stream(void* p, T v) {
  __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
}

// The lower or upper BF16 of a pair.
__device__ __forceinline__ float half_of(uint32_t pair, int upper) {
  return __builtin_bit_cast(float, upper ? pair & 0xFFFF0000u : pair << 16);
}
// Rounded to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ F8 unpack8(u32x4 p) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = half_of(p[i / 2], i & 1);
  return r;
}
__device__ __forceinline__ u32x4 pack8(const F8& f) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2((f32x2){f.v[2 * i], f.v[2 * i + 1]});
  return r;
}

__device__ __forceinline__ F8 load_f8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store_f8(float* p, const F8& f) {
  *reinterpret_cast<f32x4*>(p) = (f32x4){f.v[0], f.v[1], f.v[2], f.v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = (f32x4){f.v[4], f.v[5], f.v[6], f.v[7]};
}

// Sum over the wave, in every lane: rotations within each row of 16 lanes,
// then the four rows' sums as scalars.
template <int N>
__device__ __forceinline__ float add_ror16(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF,
                                                                   false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_ror16<8>(v);
  v = add_ror16<4>(v);
  v = add_ror16<2>(v);
  v = add_ror16<1>(v);
  float row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    row[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * i));
  return (row[0] + row[1]) + (row[2] + row[3]);
}

// v rotated by N lanes within each row of 16 lanes (DPP row_ror).
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
// Lane N of each row of 16 lanes, in all of them (DPP row_newbcast).
template <int N>
__device__ __forceinline__ int bcast16(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x150 + N, 0xF, 0xF, false);
}
// Largest over the 16 lanes of a row, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, ror16<8>(v));
  v = max(v, ror16<4>(v));
  v = max(v, ror16<2>(v));
  return max(v, ror16<1>(v));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t abs_top(const F8& x) {
  uint32_t top = abs_bits(x.v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max(top, abs_bits(x.v[i]));
  return top;
}

// The scale of a 128-value block from the largest bit pattern of its |x|:
//   scale = max(amax, 1e-4) / 448, rounded up to a power of two with E8.
// Patterns order like the values, infinity above every number and NaN above
// infinity, so a NaN anywhere gives a NaN scale.
template <bool E8>
__device__ __forceinline__ float block_scale(uint32_t top) {
  // amax / 448, correctly rounded: the product with 1/448 and one correction
  // (infinity and NaN pass through the product alone).
  const float amax = __builtin_bit_cast(float, max(top, 0x38D1B717u));  // 1e-4f
  const float near = amax * (1.0f / 448.0f);
  float scale = __builtin_fmaf(__builtin_fmaf(-near, 448.0f, amax), 1.0f / 448.0f, near);
  if (top >= 0x7F800000u) scale = near;
  if constexpr (E8) {
    // Up to a power of two: past the mantissa, then cut (finite scales only).
    const uint32_t s = __builtin_bit_cast(uint32_t, scale);
    if (s < 0x7F800000u) return __builtin_bit_cast(float, (s + 0x7FFFFFu) & 0xFF800000u);
  }
  return scale;
}

// E4M3 codes of 8 values over their block's scale. x / scale is x * (1 / scale)
// with one correction step, q + (x - q * scale) / scale, which gives the
// correctly rounded quotient: codes at a rounding tie come out as the
// division's. It needs no clamp: |x| <= amax, so |x / scale| is at most 448
// but for the rounding of the scale (448 (1 + 2^-23)), which the conversion
// rounds to 448.
__device__ __forceinline__ u32x2 quantize8(const F8& x, uint32_t top, float scale, float inv) {
  F8 q;
#pragma unroll
  for (int i = 0; i < 8; ++i) q.v[i] = x.v[i] * inv;
  if (top < 0x7F800000u) {  // else the scale is not finite and 1 / scale is 0 or NaN: so are the codes
#pragma unroll
    for (int i = 0; i < 8; ++i) q.v[i] = __builtin_fmaf(__builtin_fmaf(-q.v[i], scale, x.v[i]), inv, q.v[i]);
  }
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[4 * i], q.v[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[4 * i + 2], q.v[4 * i + 3], w, true);
    r[i] = (uint32_t)w;
  }
  return r;
}

// A block held by a row of 16 lanes, 8 values a lane.
template <bool E8>
__device__ __forceinline__ u32x2 quantize_row(const F8& x, float& scale) {
  const uint32_t top = max16(abs_top(x));
  scale = block_scale<E8>(top);
  return quantize8(x, top, scale, 1.0f / scale);
}

// Threads (a multiple of 64 up to `most`) of a workgroup that goes over `pieces`
// of work by itself: the fewest passes, and the fewest threads for those.
inline int pass_threads(int pieces, int most) {
  const int passes = (pieces + most - 1) / most;
  return ((pieces + passes - 1) / passes + 63) / 64 * 64;
}

}  // namespace moe
}  // namespace dg
