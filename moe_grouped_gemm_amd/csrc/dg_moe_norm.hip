// The norms before and after a block, fused with its gate and the residual
// scale, and their gradient.

#include <algorithm>
#include <type_traits>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

constexpr int MAX_THREADS = 1024;

// Gate values of 8 columns of a row (column gates: `channel` already holds them).
__device__ __forceinline__ F8 gate8(const void* gate, int kind, size_t t, size_t c, size_t hidden) {
  if (kind == DG_MOE_GATE_CHANNEL) return load_f8(static_cast<const float*>(gate) + c);
  if (kind == DG_MOE_GATE_FULL) return unpack8(load16(static_cast<const uint16_t*>(gate) + t * hidden + c));
  const float v = kind == DG_MOE_GATE_TOKEN ? static_cast<const float*>(gate)[t] : 1.0f;
  return F8{{v, v, v, v, v, v, v, v}};
}

// One workgroup a row, held in registers: VPT pieces of 8 columns a thread.
template <int VPT>
__global__ __launch_bounds__(MAX_THREADS) void block_norm_kernel(NormArgs p) {
  __shared__ float scratch[2][MAX_THREADS / 64];
  const size_t t = blockIdx.x, H = p.hidden;
  const int waves = blockDim.x >> 6;
  const float inv_hidden = 1.0f / (float)p.hidden;
  F8 h[VPT];
  auto column = [&](int i) { return ((size_t)i * blockDim.x + threadIdx.x) * 8; };
  if (p.y) {
    F8 y[VPT];
    float rstd = 1.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      y[i] = F8{};
      if (column(i) < H) y[i] = unpack8(load16(p.y + t * H + column(i)));
    }
    if (p.post_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(y[i].v[e], y[i].v[e], ss);
      rstd = rsqrtf(block_sum(ss, scratch[0], waves) * inv_hidden + p.eps);
      if (p.rstd_post && threadIdx.x == 0) p.rstd_post[t] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      h[i] = F8{};
      if (column(i) < H) {
        const F8 x = unpack8(load16(p.x + t * H + column(i)));
        const F8 gate = gate8(p.gate, p.gate_kind, t, column(i), H);
        F8 w = {{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
        if (p.post_weight) w = load_f8(p.post_weight + column(i));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[i].v[e] = __builtin_fmaf(p.residual_scale, x.v[e], gate.v[e] * (y[i].v[e] * rstd * w.v[e]));
        store16(p.h + t * H + column(i), pack8(h[i]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      h[i] = F8{};
      if (column(i) < H) h[i] = unpack8(load16(p.x + t * H + column(i)));
    }
  }
  if (!p.n) return;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i].v[e], h[i].v[e], ss);
  const float rstd = rsqrtf(block_sum(ss, scratch[1], waves) * inv_hidden + p.eps);
  if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[t] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (column(i) < H) {
      const F8 w = load_f8(p.pre_weight + column(i));
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i].v[e] = h[i].v[e] * rstd * w.v[e];
      store16(p.n + t * H + column(i), pack8(h[i]));
    }
  }
}

// The gradient: each workgroup takes rows in turn, keeps the sums over its
// rows of the column gradients in registers, and leaves them as one row of
// partial sums for column_sums_kernel.
template <int VPT>
__global__ __launch_bounds__(MAX_THREADS) void block_norm_bwd_kernel(NormBwdArgs p) {
  __shared__ float scratch[4][MAX_THREADS / 64];
  const size_t H = p.hidden;
  const int waves = blockDim.x >> 6;
  const float inv_hidden = 1.0f / (float)p.hidden;
  auto column = [&](int i) { return ((size_t)i * blockDim.x + threadIdx.x) * 8; };
  F8 dpost[VPT] = {}, dgate[VPT] = {}, dpre[VPT] = {};
  int turn = 0;
  for (size_t t = blockIdx.x; t < (size_t)p.tokens; t += gridDim.x, turn ^= 1) {
    F8 dres[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      dres[i] = F8{};
      if (p.dh && column(i) < H) dres[i] = unpack8(load16(p.dh + t * H + column(i)));
    }
    if (p.dn) {
      const float rstd = p.rstd_pre[t];
      F8 a[VPT], hn[VPT];
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        a[i] = hn[i] = F8{};
        if (column(i) < H) {
          const F8 dn = unpack8(load16(p.dn + t * H + column(i)));
          const F8 h = unpack8(load16(p.h + t * H + column(i)));
          const F8 w = load_f8(p.pre_weight + column(i));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hn[i].v[e] = h.v[e] * rstd;
            a[i].v[e] = dn.v[e] * w.v[e];
            dpre[i].v[e] = __builtin_fmaf(dn.v[e], hn[i].v[e], dpre[i].v[e]);
            s = __builtin_fmaf(a[i].v[e], hn[i].v[e], s);
          }
        }
      }
      const float mean = block_sum(s, scratch[turn], waves) * inv_hidden;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dres[i].v[e] = __builtin_fmaf(rstd, __builtin_fmaf(-hn[i].v[e], mean, a[i].v[e]), dres[i].v[e]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (column(i) < H) {
        F8 dx;
#pragma unroll
        for (int e = 0; e < 8; ++e) dx.v[e] = p.residual_scale * dres[i].v[e];
        store16(p.dx + t * H + column(i), pack8(dx));
      }
    }
    if (!p.y) continue;
    const float rstd = p.post_weight ? p.rstd_post[t] : 1.0f;
    F8 b[VPT], yn[VPT];
    float s = 0.f, token_gate = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      b[i] = yn[i] = F8{};
      if (column(i) < H) {
        const F8 y = unpack8(load16(p.y + t * H + column(i)));
        const F8 gate = gate8(p.gate, p.gate_kind, t, column(i), H);
        F8 w = {{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
        if (p.post_weight) w = load_f8(p.post_weight + column(i));
        F8 dg;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yn[i].v[e] = y.v[e] * rstd;
          dg.v[e] = dres[i].v[e] * (yn[i].v[e] * w.v[e]);
          const float dp = dres[i].v[e] * gate.v[e];
          dpost[i].v[e] = __builtin_fmaf(dp, yn[i].v[e], dpost[i].v[e]);
          dgate[i].v[e] += dg.v[e];
          token_gate += dg.v[e];
          b[i].v[e] = dp * w.v[e];
          s = __builtin_fmaf(b[i].v[e], yn[i].v[e], s);
        }
        if (p.gate_kind == DG_MOE_GATE_FULL && p.dgate)
          store16(static_cast<uint16_t*>(p.dgate) + t * H + column(i), pack8(dg));
      }
    }
    if (p.gate_kind == DG_MOE_GATE_TOKEN && p.dgate) {
      token_gate = block_sum(token_gate, scratch[turn], waves);
      if (threadIdx.x == 0) static_cast<float*>(p.dgate)[t] = token_gate;
    }
    float mean = 0.f;
    if (p.post_weight) mean = block_sum(s, scratch[2 + turn], waves) * inv_hidden;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (column(i) < H) {
        F8 dy;
#pragma unroll
        for (int e = 0; e < 8; ++e) dy.v[e] = rstd * __builtin_fmaf(-yn[i].v[e], mean, b[i].v[e]);
        store16(p.dy + t * H + column(i), pack8(dy));
      }
    }
  }
  float* out = p.partial + (size_t)blockIdx.x * 3 * H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (column(i) < H) {
      store_f8(out + column(i), dpost[i]);
      store_f8(out + H + column(i), dgate[i]);
      store_f8(out + 2 * H + column(i), dpre[i]);
    }
  }
}

// Sums the partial rows, in order: the result does not depend on timing.
__global__ __launch_bounds__(64) void column_sums_kernel(NormBwdArgs p, int parts) {
  const int c = blockIdx.x * 64 + threadIdx.x, which = blockIdx.y;
  float* out = which == 0 ? p.dpost
               : which == 1 ? (p.gate_kind == DG_MOE_GATE_CHANNEL ? static_cast<float*>(p.dgate) : nullptr)
                            : p.dpre;
  if (!out || c >= p.hidden) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += p.partial[((size_t)i * 3 + which) * p.hidden + c];
  out[c] = s;
}

// Threads and pieces a thread for a row of `hidden` values.
void row_shape(int hidden, int& threads, int& vpt) {
  const int pieces = hidden / 8;
  vpt = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
  threads = ((pieces + vpt - 1) / vpt + 63) / 64 * 64;
}

template <class F>
void with_vpt(int vpt, F&& f) {
  if (vpt == 1) f(std::integral_constant<int, 1>{});
  else if (vpt == 2) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 4>{});
}

}  // namespace

int norm_bwd_grid(int tokens, int hidden) {
  (void)hidden;
  return std::min(tokens, 256);
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream) {
  int threads, vpt;
  row_shape(a.hidden, threads, vpt);
  with_vpt(vpt, [&](auto v) {
    hipLaunchKernelGGL(block_norm_kernel<decltype(v)::value>, dim3(a.tokens), dim3(threads), 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  int threads, vpt;
  row_shape(a.hidden, threads, vpt);
  const int grid = norm_bwd_grid(a.tokens, a.hidden);
  if (grid > 0) {
    with_vpt(vpt, [&](auto v) {
      hipLaunchKernelGGL(block_norm_bwd_kernel<decltype(v)::value>, dim3(grid), dim3(threads), 0, stream, a);
    });
    if (hipError_t e = hipGetLastError()) return e;
  }
  hipLaunchKernelGGL(column_sums_kernel, dim3((a.hidden + 63) / 64, 3), dim3(64), 0, stream, a, grid);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
