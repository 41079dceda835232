// The norms before and after a block, fused with its gate and the residual
// scale, and their gradient.
//
// A row is held in registers by a team of 1 to 16 waves, VPT pieces of 8
// columns a lane; a workgroup holds as many teams as fit 1024 threads, and
// takes rows in turn. Column vectors (weights, a channel gate) are the same
// for every row: with one piece a lane they stay in registers for all of the
// workgroup's rows (read per row they would be more L2 traffic than the rows
// themselves: 3 x 4 bytes a column against 2 x 2). Later rows' loads are issued
// while a row is worked on, so the sums a row needs (wave sums, joined through LDS
// where the team has more waves) run under them. Bound by memory: every
// activation is read once and written once. 8192 rows of 7168: 82 us forward (470
// MB, 5.7 TB/s); the gradient of 4099 rows: 72 us with its column sums (353 MB).
// Other figures here are ratios, or of other sizes.

#include <algorithm>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

typedef dg_moe_norm NormArgs;
typedef dg_moe_norm_bwd NormBwdArgs;  // workspace: [workgroups][2][hidden] float32, sums over rows of dH yn and dn hn

constexpr int MAX_THREADS = 1024;
constexpr int MAX_WAVES = MAX_THREADS / 64;

// How a workgroup shares rows: teams of `waves` waves.
struct TeamShape {
  int waves, teams, vpt;
  int threads() const { return waves * teams * 64; }
};

// Where this thread stands.
struct Team {
  int waves, first_wave, lane_in_team;
  int team, teams;
};
__device__ __forceinline__ Team team_of(int waves) {
  // the same in all lanes of a wave: rows' addresses stay in scalar registers
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / waves;
  return {waves, team * waves, (int)threadIdx.x - team * waves * 64, team, (int)(blockDim.x >> 6) / waves};
}

// Sum over the team, in every lane. Every wave of the workgroup calls it the
// same number of times; `scratch` may be written again after a later barrier.
// The waves' sums are read 16 at once, one a lane, and added by rotations: a
// loop over them would wait for LDS once a wave.
__device__ __forceinline__ float row_sum(float v) {
  return add_ror16<1>(add_ror16<2>(add_ror16<4>(add_ror16<8>(v))));
}
__device__ __forceinline__ float team_sum(float v, const Team& tm, float* scratch) {
  v = wave_sum(v);
  if (tm.waves == 1) return v;
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  const int w = threadIdx.x & 15;
  return row_sum(w < tm.waves ? scratch[tm.first_wave + w] : 0.f);
}

__device__ __forceinline__ F8 splat(float v) { return F8{{v, v, v, v, v, v, v, v}}; }

// A row's pieces as loaded.
template <int VPT>
__device__ __forceinline__ void load_row(u32x4 (&out)[VPT], const void* base, size_t t, int hidden, const Team& tm,
                                         bool live) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * tm.waves * 64 + tm.lane_in_team) * 8;
    out[i] = (u32x4){0, 0, 0, 0};
    if (live && base && c < hidden) out[i] = load_stream16(static_cast<const uint16_t*>(base) + t * hidden + c);
  }
}

// A column vector's values at this thread's columns: kept (one piece a lane)
// or read when asked for.
template <int VPT>
struct Column {
  F8 kept;
  const float* base;
  __device__ __forceinline__ void init(const float* p, int c, int hidden, float none) {
    base = p;
    kept = splat(none);
    if (VPT == 1 && p && c < hidden) kept = load_f8(p + c);
  }
  __device__ __forceinline__ F8 at(int c, int hidden) const {
    if (VPT == 1 || !base || c >= hidden) return kept;
    return load_f8(base + c);
  }
};

template <int VPT>
__global__ __launch_bounds__(MAX_THREADS) void block_norm_kernel(NormArgs p, int waves) {
  __shared__ float scratch[4][MAX_WAVES];
  const Team tm = team_of(waves);
  const int H = p.hidden;
  const float inv_hidden = 1.0f / (float)H;
  const bool full_gate = p.gate_kind == DG_MOE_GATE_FULL;
  Column<VPT> post, pre, gate;
  const int c0 = tm.lane_in_team * 8;
  post.init(p.post_weight, c0, H, 1.0f);
  pre.init(p.pre_weight, c0, H, 1.0f);
  gate.init(p.gate_kind == DG_MOE_GATE_CHANNEL ? static_cast<const float*>(p.gate) : nullptr, c0, H, 1.0f);

  const int step = gridDim.x * tm.teams;
  int t = blockIdx.x + gridDim.x * tm.team;
  const int rounds = (p.tokens + step - 1) / step;
  u32x4 x[VPT], y[VPT], g[VPT];
  float next_gate = 1.0f;
  auto load = [&](int row) {
    const bool live = row < p.tokens;
    if (p.gate_kind == DG_MOE_GATE_TOKEN && live) next_gate = static_cast<const float*>(p.gate)[row];
    load_row(x, p.x, row, H, tm, live);
    load_row(y, p.y, row, H, tm, live);
    if (full_gate) load_row(g, p.gate, row, H, tm, live);
  };
  load(t);
  for (int round = 0; round < rounds; ++round, t += step) {
    float* s0 = scratch[2 * (round & 1)];
    const bool live = t < p.tokens;
    const float row_gate = next_gate;
    F8 h[VPT];
    if (p.y) {
      float rstd = 1.0f;
      if (p.post_weight) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const F8 v = unpack8(y[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v.v[e], v.v[e], ss);
        }
        rstd = rsqrtf(team_sum(ss, tm, s0) * inv_hidden + p.eps);
        if (p.rstd_post && live && tm.lane_in_team == 0) p.rstd_post[t] = rstd;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * waves * 64 + tm.lane_in_team) * 8;
        const F8 xv = unpack8(x[i]), yv = unpack8(y[i]), w = post.at(c, H);
        const F8 gv = full_gate ? unpack8(g[i]) : gate.at(c, H);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[i].v[e] = __builtin_fmaf(p.residual_scale, xv.v[e], row_gate * gv.v[e] * (yv.v[e] * rstd * w.v[e]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) h[i] = unpack8(x[i]);
    }
    // The next row is asked for once this one has been read out; asked for
    // earlier it would come before this row's own waits (a seventh slower).
    load(t + step);
    if (p.y) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * waves * 64 + tm.lane_in_team) * 8;
        if (live && c < H) store_stream(static_cast<uint16_t*>(p.h) + (size_t)t * H + c, pack8(h[i]));
      }
    }
    if (!p.n) continue;
    // Pieces past the row were loaded as zeros, but an infinite gate or factor makes NaN of them.
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if ((i * waves * 64 + tm.lane_in_team) * 8 >= H) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i].v[e], h[i].v[e], ss);
    }
    const float rstd = rsqrtf(team_sum(ss, tm, s0 + MAX_WAVES) * inv_hidden + p.eps);
    if (p.rstd_pre && live && tm.lane_in_team == 0) p.rstd_pre[t] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * waves * 64 + tm.lane_in_team) * 8;
      const F8 w = pre.at(c, H);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i].v[e] = h[i].v[e] * rstd * w.v[e];
      if (live && c < H) store_stream(static_cast<uint16_t*>(p.n) + (size_t)t * H + c, pack8(h[i]));
    }
  }
}

// The gradient. With hn = h rstd_pre, a = dn pre_weight, yn = y rstd_post and v
// the weight that meets a row's dH on the way to y (gate * post_weight, without
// the token gate, which multiplies a whole row):
//     dH = dh + rstd_pre (a - hn m),  m = mean(a hn)
//     dy = rstd_post token_gate (dH v - yn mean(dH v yn))
// and sum(dH v yn) = sum((dh + rstd_pre a) v yn) - rstd_pre m sum(hn v yn), so all
// of a row's sums are taken at once, from its inputs alone: one barrier a row.
// The column gradients need one sum besides dpre_weight's: a channel gate and
// post_weight are the same for every row, so both of their gradients are
// S = sum_t dH yn times the other one (with token or full gates inside S,
// dpost_weight is S itself). They are summed over the team's rows in
// registers; at the end the teams' sums are added up in LDS, in order, and
// leave the workgroup as one row of partial sums for column_sums_kernel.
template <int VPT, bool FULL>
__global__ __launch_bounds__(MAX_THREADS) void block_norm_bwd_kernel(NormBwdArgs p, int waves) {
  __shared__ f32x4 scratch[2][MAX_WAVES];
  // The column vectors in LDS where they do not fit the registers beside a full
  // gate or a second piece a lane: to y, then to h. (Read from global memory in
  // the loop they would wait for the next row's loads, issued before them.) At the
  // end the same memory takes the teams' column sums, [2][hidden]; several teams
  // have a hidden of at most 4096.
  constexpr bool IN_LDS = FULL || VPT > 1;
  constexpr int MOST = MAX_THREADS * 8 * VPT;
  __shared__ __align__(16) float columns[IN_LDS ? 2 * MOST : MOST];
  const Team tm = team_of(waves);
  const int H = p.hidden;
  const float inv_hidden = 1.0f / (float)H;
  const float* channel = p.gate_kind == DG_MOE_GATE_CHANNEL ? static_cast<const float*>(p.gate) : nullptr;
  auto column = [&](int i) { return (i * waves * 64 + tm.lane_in_team) * 8; };
  // v without a full gate, and pre_weight, at a piece's columns.
  auto to_y = [&](int c) {
    F8 v = splat(1.0f);
    if (c < H) {
      if (p.post_weight) v = load_f8(p.post_weight + c);
      if (channel) {
        const F8 g = load_f8(channel + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] *= g.v[e];
      }
    }
    return v;
  };
  auto to_h = [&](int c) { return p.pre_weight && c < H ? load_f8(p.pre_weight + c) : splat(1.0f); };
  F8 keep_y, keep_h;
  if constexpr (IN_LDS) {
    for (int c = threadIdx.x * 8; c < VPT * waves * 512; c += blockDim.x * 8) {
      store_f8(columns + c, to_y(c));
      store_f8(columns + MOST + c, to_h(c));
    }
    __syncthreads();
  } else {
    keep_y = to_y(column(0));
    keep_h = to_h(column(0));
  }
  // Of pair q of piece i's columns.
  auto weight_y = [&](int i, int q) {
    if constexpr (IN_LDS) return *reinterpret_cast<const f32x2*>(columns + column(i) + 2 * q);
    else return (f32x2){keep_y.v[2 * q], keep_y.v[2 * q + 1]};
  };
  auto weight_h = [&](int i, int q) {
    if constexpr (IN_LDS) return *reinterpret_cast<const f32x2*>(columns + MOST + column(i) + 2 * q);
    else return (f32x2){keep_h.v[2 * q], keep_h.v[2 * q + 1]};
  };
  F8 dpost[VPT] = {}, dpre[VPT] = {};

  const int step = gridDim.x * tm.teams;
  int t = blockIdx.x + gridDim.x * tm.team;
  const int rounds = (p.tokens + step - 1) / step;
  struct Row {
    u32x4 dh[VPT], dn[VPT], h[VPT], y[VPT], g[FULL ? VPT : 1];
    float rstd_pre, rstd_post, gate;
  };
  auto load = [&](Row& r, int row) {
    const bool live = row < p.tokens;
    r.rstd_pre = live && p.dn ? p.rstd_pre[row] : 0.0f;
    r.rstd_post = live && p.post_weight ? p.rstd_post[row] : 1.0f;
    r.gate = live && p.gate_kind == DG_MOE_GATE_TOKEN ? static_cast<const float*>(p.gate)[row] : 1.0f;
    load_row(r.dn, p.dn, row, H, tm, live);
    load_row(r.h, p.dn ? p.h : nullptr, row, H, tm, live);
    load_row(r.dh, p.dh, row, H, tm, live);
    load_row(r.y, p.y, row, H, tm, live);
    if constexpr (FULL) load_row<VPT>(r.g, p.gate, row, H, tm, live);
  };
  // Two rows on their way where the registers allow, else one or none: 4099 rows of
  // 7168 take 4% less time with two than with one.
  constexpr int LEAD = VPT > 1 ? 0 : FULL ? 1 : 2;
  Row ahead[2];
  if constexpr (LEAD > 0) load(ahead[0], t);
  if constexpr (LEAD > 1) load(ahead[1], t + step);
  for (int round = 0; round < rounds; ++round, t += step) {
    const bool live = t < p.tokens;
    Row r;
    if constexpr (LEAD == 0) {
      load(r, t);
    } else {
      r = ahead[0];
      if constexpr (LEAD > 1) ahead[0] = ahead[1];
      load(ahead[LEAD - 1], t + LEAD * step);
    }
    float s_a = 0.f, s_b = 0.f, s_c = 0.f;  // of a h, (dh + rstd_pre a) v y, h v y: the rstd factors follow
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x2 w2 = weight_h(i, q), v2 = weight_y(i, q);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float h = half_of(r.h[i][q], e);
          const float a = half_of(r.dn[i][q], e) * w2[e];
          float vy = v2[e] * half_of(r.y[i][q], e);
          if constexpr (FULL) vy *= half_of(r.g[i][q], e);
          s_a = __builtin_fmaf(a, h, s_a);
          s_b = __builtin_fmaf(__builtin_fmaf(r.rstd_pre, a, half_of(r.dh[i][q], e)), vy, s_b);
          s_c = __builtin_fmaf(h, vy, s_c);
        }
        if constexpr (IN_LDS) __builtin_amdgcn_sched_barrier(0);
      }
    }
    s_a = wave_sum(s_a);
    s_b = wave_sum(s_b);
    s_c = wave_sum(s_c);
    if (waves > 1) {
      f32x4* s = scratch[round & 1];
      if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = (f32x4){s_a, s_b, s_c, 0.f};
      __syncthreads();
      const int w = threadIdx.x & 15;
      f32x4 part = {0.f, 0.f, 0.f, 0.f};
      if (w < waves) part = s[tm.first_wave + w];
      s_a = row_sum(part[0]);
      s_b = row_sum(part[1]);
      s_c = row_sum(part[2]);
    }
    // dH = (dh + rstd_pre a) + to_dres h; sum of dH v yn; dy = out dH v + to_dy y
    const float to_dres = -(s_a * r.rstd_pre * inv_hidden) * r.rstd_pre * r.rstd_pre;
    const float along = r.rstd_post * __builtin_fmaf(to_dres, s_c, s_b);
    const float mean = p.post_weight ? along * inv_hidden : 0.0f;
    if (p.gate_kind == DG_MOE_GATE_TOKEN && p.dgate && live && tm.lane_in_team == 0)
      static_cast<float*>(p.dgate)[t] = along;
    const float out = r.rstd_post * r.gate, to_dy = -(out * mean) * r.rstd_post;
    // The pieces are unpacked again rather than kept as floats across the
    // sums: those would not fit the registers, and a spilled value's reload
    // waits for the next row's loads, which were issued before it.
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      asm volatile("" : "+v"(r.dn[i]), "+v"(r.h[i]), "+v"(r.dh[i]), "+v"(r.y[i]));
      if constexpr (FULL) asm volatile("" : "+v"(r.g[i]));
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column(i);
      u32x4 dx, dy, dg;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x2 w2 = weight_h(i, q), v2 = weight_y(i, q);
        f32x2 dx2, dy2, dg2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float h = half_of(r.h[i][q], e), y = half_of(r.y[i][q], e);
          const float dr = half_of(r.dn[i][q], e) * r.rstd_pre;
          const float dres = __builtin_fmaf(to_dres, h, __builtin_fmaf(dr, w2[e], half_of(r.dh[i][q], e)));
          dpre[i].v[2 * q + e] = __builtin_fmaf(dr, h, dpre[i].v[2 * q + e]);
          dx2[e] = p.residual_scale * dres;
          float gated = dres, to = dres * v2[e];
          if constexpr (FULL) {
            const float g = half_of(r.g[i][q], e);
            dg2[e] = to * (y * r.rstd_post);
            gated *= g;
            to *= g;
          }
          dpost[i].v[2 * q + e] = __builtin_fmaf(gated, y * out, dpost[i].v[2 * q + e]);
          dy2[e] = __builtin_fmaf(out, to, to_dy * y);
        }
        dx[q] = pack2(dx2);
        dy[q] = pack2(dy2);
        if constexpr (FULL) dg[q] = pack2(dg2);
        if constexpr (IN_LDS) __builtin_amdgcn_sched_barrier(0);  // as few registers at once as can be
      }
      if (live && c < H) {
        store_stream(static_cast<uint16_t*>(p.dx) + (size_t)t * H + c, dx);
        if (p.y) store_stream(static_cast<uint16_t*>(p.dy) + (size_t)t * H + c, dy);
        if (FULL && p.dgate) store_stream(static_cast<uint16_t*>(p.dgate) + (size_t)t * H + c, dg);
      }
    }
  }

  float* out = static_cast<float*>(p.workspace) + (size_t)blockIdx.x * 2 * H;
  if (IN_LDS && tm.teams > 1) __syncthreads();
  for (int turn = 0; turn < tm.teams; ++turn) {
    if (turn > 0) __syncthreads();
    if (turn != tm.team) continue;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column(i);
      if (c >= H) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        F8 v = k == 0 ? dpost[i] : dpre[i];
        if (turn > 0) {
          const F8 before = load_f8(columns + k * H + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) v.v[e] += before.v[e];
        }
        if (turn + 1 < tm.teams) store_f8(columns + k * H + c, v);
        else store_f8(out + k * H + c, v);
      }
    }
  }
}

// Sums the partial rows in a fixed order: the result does not depend on
// timing. 64 columns a workgroup, 16 threads across (4 columns each) and 16
// down, each down thread every 16th row: 256 rows of 2 x 7168 in 5.3 us (2.8 TB/s),
// bound by latency; a thread a column took 61. 32 and 64 down were no faster.
__global__ __launch_bounds__(256) void column_sums_kernel(NormBwdArgs p, int parts) {
  __shared__ f32x4 down[16][16];
  const int across = threadIdx.x & 15, row = threadIdx.x >> 4;
  const bool pre = blockIdx.y == 1;
  const int c = blockIdx.x * 64 + across * 4;
  const float* channel = p.gate_kind == DG_MOE_GATE_CHANNEL ? static_cast<const float*>(p.gate) : nullptr;
  float* dgate = channel ? static_cast<float*>(p.dgate) : nullptr;
  if (pre ? !p.dpre_weight : !p.dpost_weight && !dgate) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < p.hidden) {
#pragma unroll 8
    for (int i = row; i < parts; i += 16)
      s += *reinterpret_cast<const f32x4*>(static_cast<float*>(p.workspace) + ((size_t)i * 2 + pre) * p.hidden + c);
  }
  down[row][across] = s;
  __syncthreads();
  if (row == 0 && c < p.hidden) {
    for (int i = 1; i < 16; ++i) s += down[i][across];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (pre) {
        p.dpre_weight[c + i] = s[i];
      } else {
        if (p.dpost_weight) p.dpost_weight[c + i] = s[i] * (channel ? channel[c + i] : 1.0f);
        if (dgate) dgate[c + i] = s[i] * (p.post_weight ? p.post_weight[c + i] : 1.0f);
      }
    }
  }
}

constexpr int MOST_WORKGROUPS = 256;  // the device's CUs

// As many teams as a workgroup has room and rows for: waves without rows make
// every launch longer, and each team is a turn at the gradient's end (512 rows of
// 512: 3.0 us forward and 8.0 back, with 16 teams 4.1 and 12.2).
TeamShape team_shape(int tokens, int hidden, int grid) {
  const int pieces = hidden / 8, vpt = pieces <= MAX_THREADS ? 1 : 2;
  const int waves = ((pieces + vpt - 1) / vpt + 63) / 64;
  return {waves, std::min(MAX_WAVES / waves, (tokens + grid - 1) / grid), vpt};
}

// One workgroup a CU of the `cus` that the caller leaves the kernels: 2 and 4 are
// slower (8192 rows of 7168 by 3 and 7%, the gradient of 4099 rows by 12 and 36%).
// Fewer where they need no more rounds of rows are no faster: a round takes what a
// CU takes for its rows.
int row_grid(int tokens, int cus) { return std::min({tokens, cus, MOST_WORKGROUPS}); }

}  // namespace

int norm_bwd_grid(int tokens) { return row_grid(tokens, MOST_WORKGROUPS); }

hipError_t launch_block_norm(const NormArgs& a, int cus, hipStream_t stream) {
  const int grid = row_grid(a.tokens, cus);
  const TeamShape s = team_shape(a.tokens, a.hidden, grid);
  auto* kernel = s.vpt == 1 ? block_norm_kernel<1> : block_norm_kernel<2>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(s.threads()), 0, stream, a, s.waves);
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(const NormBwdArgs& a, int cus, hipStream_t stream) {
  const int grid = row_grid(a.tokens, cus);
  if (grid > 0) {
    const TeamShape s = team_shape(a.tokens, a.hidden, grid);
    const bool full = a.gate_kind == DG_MOE_GATE_FULL;
    auto* kernel = s.vpt == 1 ? (full ? block_norm_bwd_kernel<1, true> : block_norm_bwd_kernel<1, false>)
                              : (full ? block_norm_bwd_kernel<2, true> : block_norm_bwd_kernel<2, false>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(s.threads()), 0, stream, a, s.waves);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!a.dpost_weight && !a.dpre_weight && !(a.gate_kind == DG_MOE_GATE_CHANNEL && a.dgate)) return hipSuccess;
  hipLaunchKernelGGL(column_sums_kernel, dim3((a.hidden + 63) / 64, 2), dim3(256), 0, stream, a, grid);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
