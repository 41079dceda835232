// Rows quantised to the FP4 GEMMs' operands (E2M1 codes with one E8M0 scale per
// 32 values, the four scales of 128 values in one word) and read back.
//
// A workgroup takes 32 rows of 512 values, 16 lanes a 128-value block (a scale's
// 32 values are 4 lanes, the largest by two DPP permutations) and a row's four
// blocks' loads on their way at once. The words of 32 rows, which lie side by
// side, leave as one 128-byte line a block. Bound by memory: 8 x 4096 x 7168 from
// float32 in 197 us, 5.4 TB/s (a copy runs at 5.0), read back in 100, 5.9 TB/s.

#include <algorithm>

#include "dg_internal.h"
#include "dg_moe_device.h"

namespace dg {
namespace {

using namespace moe;

constexpr int TILE_ROWS = 32, TILE_BLOCKS = 4, TILE_THREADS = TILE_ROWS * 16;

// Calls f(group, first row, first block) for each of the workgroup's tiles.
template <class F>
__device__ __forceinline__ void for_tiles(int groups, int rows, int blocks, F&& f) {
  const uint32_t across = (blocks + TILE_BLOCKS - 1) / TILE_BLOCKS, down = (rows + TILE_ROWS - 1) / TILE_ROWS;
  const uint64_t tiles = (uint64_t)groups * down * across;
  for (uint64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint32_t b = (uint32_t)(t % across), r = (uint32_t)(t / across);  // (below 2^31: rows take memory)
    f((int)(r / down), (int)(r % down) * TILE_ROWS, (int)b * TILE_BLOCKS);
  }
}

template <bool WIDE>
__global__ __launch_bounds__(TILE_THREADS) void quantize_fp4_kernel(QuantizeArgs p) {
  __shared__ uint32_t words[TILE_BLOCKS][TILE_ROWS];
  const int team = threadIdx.x >> 4, l16 = threadIdx.x & 15, blocks = p.k / QBLOCK;
  for_tiles(p.groups, p.rows, blocks, [&](int g, int r0, int b0) {
    const int here = min(blocks - b0, TILE_BLOCKS);
    if (r0 + team < p.rows) {
      const size_t row = (size_t)g * p.rows + r0 + team, at = row * p.k + (size_t)b0 * QBLOCK + l16 * 8;
      u32x4 raw[TILE_BLOCKS][WIDE ? 2 : 1];
#pragma unroll
      for (int b = 0; b < TILE_BLOCKS; ++b)
        if (b < here) {
          if constexpr (WIDE) {
            const float* src = static_cast<const float*>(p.x) + at + b * QBLOCK;
            raw[b][0] = load_stream16(src);
            raw[b][1] = load_stream16(src + 4);
          } else {
            raw[b][0] = load_stream16(static_cast<const uint16_t*>(p.x) + at + b * QBLOCK);
          }
        }
#pragma unroll
      for (int b = 0; b < TILE_BLOCKS; ++b)
        if (b < here) {
          F8 x;
          if constexpr (WIDE) {
            const f32x4 lo = __builtin_bit_cast(f32x4, raw[b][0]), hi = __builtin_bit_cast(f32x4, raw[b][1]);
            x = F8{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
          } else {
            x = unpack8(raw[b][0]);
          }
          const uint32_t code = fp4_scale(max4(abs_top(x)));
          store_stream(p.q + (at + b * QBLOCK) / 2, fp4_codes(x, code));
          const uint32_t word = fp4_scale_word(code);
          if (l16 == 0) words[b][team] = word;
        }
    }
    __syncthreads();
    const int b = threadIdx.x / TILE_ROWS, r = threadIdx.x % TILE_ROWS;
    if (b < here && r0 + r < p.rows) p.sf[((size_t)g * blocks + b0 + b) * p.ld + r0 + r] = words[b][r];
    __syncthreads();  // the words are read before the next tile's
  });
}

__global__ __launch_bounds__(TILE_THREADS) void dequantize_fp4_kernel(const uint8_t* q, const uint32_t* sf,
                                                                      uint16_t* x, int groups, int rows, int k,
                                                                      int ld) {
  const int team = threadIdx.x >> 4, l16 = threadIdx.x & 15, blocks = k / QBLOCK;
  for_tiles(groups, rows, blocks, [&](int g, int r0, int b0) {
    if (r0 + team >= rows) return;
    const int here = min(blocks - b0, TILE_BLOCKS);
    const size_t row = (size_t)g * rows + r0 + team, at = row * k + (size_t)b0 * QBLOCK + l16 * 8;
    const uint32_t* scales = sf + ((size_t)g * blocks + b0) * ld + r0 + team;
    uint32_t codes[TILE_BLOCKS], words[TILE_BLOCKS];
#pragma unroll
    for (int b = 0; b < TILE_BLOCKS; ++b)
      if (b < here) {
        codes[b] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q + (at + b * QBLOCK) / 2));
        words[b] = scales[(size_t)b * ld];
      }
#pragma unroll
    for (int b = 0; b < TILE_BLOCKS; ++b)
      if (b < here) store_stream(x + at + b * QBLOCK, fp4_values(codes[b], words[b] >> (l16 >> 2) * 8 & 0xFF));
  });
}

int tile_grid(int groups, int rows, int k) {
  const long long tiles = (long long)groups * ((rows + TILE_ROWS - 1) / TILE_ROWS) *
                          ((k / QBLOCK + TILE_BLOCKS - 1) / TILE_BLOCKS);
  return (int)std::min<long long>(tiles, 1 << 22);  // workgroups * threads stay below 2^32
}

}  // namespace

hipError_t launch_quantize_fp4(const QuantizeArgs& a, hipStream_t stream) {
  auto* kernel = a.wide ? quantize_fp4_kernel<true> : quantize_fp4_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(tile_grid(a.groups, a.rows, a.k)), dim3(TILE_THREADS), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_dequantize_fp4(const uint8_t* q, const uint32_t* sf, void* x, int groups, int rows, int k, int ld,
                                 hipStream_t stream) {
  hipLaunchKernelGGL(dequantize_fp4_kernel, dim3(tile_grid(groups, rows, k)), dim3(TILE_THREADS), 0, stream, q, sf,
                     static_cast<uint16_t*>(x), groups, rows, k, ld);
  return hipGetLastError();
}

}  // namespace dg
