// A whole expert layer for a few tokens in two launches:
//
//   a[t, e] = silu(g) * u,  [g | u] = B1[e] x[t]        (up)
//   y[t]    = sum_j w[t, j] * B2[e] a[t, e], e = ids[t, j]   (down)
//
// with the experts' weights in FP8 (one float32 scale per 128 x 128) or FP4 (one
// power-of-two scale per 32 values of a row) and everything else as it comes: x in
// BF16, sums in float32, a rounded once to BF16 (the rounding of y itself is as
// large; a grouped product's path rounds g, u and then a to FP8). The weights of
// the experts that have tokens are read once, and that bounds both launches:
// every wave streams weights from memory straight into registers, converts them to
// BF16 (exact: E4M3 has 4 significant bits, E2M1 2) and multiplies them on the
// matrix cores with up to 16 tokens a tile, whose rows come from L2.
//
// v_mfma_f32_16x16x32_bf16: the first operand's lane (r, g) = (lane % 16, lane /
// 16) holds 8 values of K of weight row r, the second's of token r, and result i of
// the lane is weight row 4g + i for token r. Lane group g takes K positions 32g ..
// 32g + 31 of 128 in four such steps, so that a lane's weights are 32 successive
// bytes (FP8) or 16 (FP4), one scale block.

#include <algorithm>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// What the first launch leaves for the second, before the activations: the experts
// that have tokens, in order of their first slot, and their (token, expert) pairs.
// A pair is known by its first slot, and its activation lies in that slot's row; a
// token that names an expert twice is one pair with the weights' sum.
struct ExpertEntry {
  int expert, begin, count, pad;
};
struct ExpertPlan {
  int experts, pairs, pad[2];
  ExpertEntry entry[MAX_FEW_PAIRS];
  int slot[MAX_FEW_PAIRS];
  float weight[MAX_FEW_PAIRS];
};
static_assert(sizeof(ExpertPlan) == EXPERT_PLAN_BYTES, "room for the plan");

// ---------------------------------------------------------------------------
// Weights
// ---------------------------------------------------------------------------

// A chunk is 128 bytes of a weight row: 128 values of FP8, 256 of FP4.
template <bool FP4>
constexpr int CHUNK_BLOCKS = FP4 ? 2 : 1;

// One expert's matrix [rows][k] and its scales.
struct Matrix {
  const uint8_t* w;
  const void* sf;  // FP8: float [rows/128][k/128]; FP4: words [k/128][ld]
  int k, ld;
};

// A 16-row tile's chunk as loaded: lane (r, g) of row r.
template <bool FP4>
struct Chunk {
  u32x4 w[2];       // FP8: bytes 32g .. + 31; FP4: bytes 16g .. + 15 of either block
  uint32_t sf[FP4 ? 2 : 1];
};

template <bool FP4>
__device__ __forceinline__ void load_chunk(Chunk<FP4>& c, const Matrix& m, int row0, int block, int lane) {
  const int r = lane & 15, g = lane >> 4, blocks = m.k / QBLOCK;
  if constexpr (FP4) {
    const uint8_t* src = m.w + (size_t)(row0 + r) * (m.k / 2) + block * 64 + g * 16;
    const uint32_t* sf = static_cast<const uint32_t*>(m.sf) + (size_t)block * m.ld + row0 + r;
    c.w[0] = load_stream16(src);
    c.sf[0] = sf[0];
    c.w[1] = (u32x4){0, 0, 0, 0};
    c.sf[1] = 0;
    if (block + 1 < blocks) {
      c.w[1] = load_stream16(src + 64);
      c.sf[1] = sf[m.ld];
    }
  } else {
    const uint8_t* src = m.w + (size_t)(row0 + r) * m.k + block * 128 + g * 32;
    c.w[0] = load_stream16(src);
    c.w[1] = load_stream16(src + 16);
    c.sf[0] = static_cast<const uint32_t*>(m.sf)[(size_t)(row0 / 128) * blocks + block];
  }
}

__device__ __forceinline__ bf16x8 as_operand(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// The four operands of one 128-value block.
template <bool FP4>
__device__ __forceinline__ void operands(const Chunk<FP4>& c, int b, int g, bf16x8 (&out)[4]) {
  if constexpr (FP4) {
    const uint32_t code = (c.sf[b] >> (8 * g)) & 0xFF;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t dword = c.w[b][j];
      out[j] = as_operand(fp4_values(dword, code));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c.w[j / 2][2 * (j & 1)], hi = c.w[j / 2][2 * (j & 1) + 1];
      const u32x4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
      out[j] = as_operand(v);
    }
  }
}

// Tokens' values of the same chunk: lane (r, g) of token r.
template <bool FP4, int NT>
struct Tokens {
  u32x4 v[NT][4 * CHUNK_BLOCKS<FP4>];
};

template <bool FP4, int NT>
__device__ __forceinline__ void load_tokens(Tokens<FP4, NT>& t, const uint16_t* const (&row)[NT], int block,
                                            int blocks, int lane) {
  const int g = lane >> 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int b = 0; b < CHUNK_BLOCKS<FP4>; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t.v[nt][4 * b + j] = (u32x4){0, 0, 0, 0};
        if (b == 0 || block + b < blocks) t.v[nt][4 * b + j] = load16(row[nt] + (block + b) * QBLOCK + 32 * g + 8 * j);
      }
}

// acc += the chunk's weights times the tokens.
template <bool FP4, int NT>
__device__ __forceinline__ void multiply(f32x4 (&acc)[NT], const Chunk<FP4>& c, const Tokens<FP4, NT>& t, int lane) {
  bf16x8 w[4];
  if constexpr (FP4) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      operands<FP4>(c, b, lane >> 4, w);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], as_operand(t.v[nt][4 * b + j]), acc[nt], 0, 0, 0);
    }
  } else {
    operands<FP4>(c, 0, lane >> 4, w);
    const float s = __builtin_bit_cast(float, c.sf[0]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], as_operand(t.v[nt][j]), part, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = __builtin_fmaf(part[i], s, acc[nt][i]);
    }
  }
}

// Sums of TILES 16-row tiles, tile i from matrix row row0[i], over the chunks
// first, first + step, ... below `end` (counted in chunks): the next chunk's
// loads are on their way while one is multiplied.
template <bool FP4, int TILES, int NT>
__device__ __forceinline__ void stream_rows(f32x4 (&acc)[TILES][NT], const Matrix& m, const int (&row0)[TILES],
                                            const uint16_t* const (&row)[NT], int first, int step, int end,
                                            int lane) {
  constexpr int CB = CHUNK_BLOCKS<FP4>;
  const int blocks = m.k / QBLOCK;
  Chunk<FP4> c[2][TILES];
  Tokens<FP4, NT> t[2];
  auto load = [&](auto S, int chunk) {
    constexpr int s = decltype(S)::value;
#pragma unroll
    for (int i = 0; i < TILES; ++i) load_chunk<FP4>(c[s][i], m, row0[i], chunk * CB, lane);
    load_tokens<FP4, NT>(t[s], row, chunk * CB, blocks, lane);
  };
  auto multiply_all = [&](auto S) {
    constexpr int s = decltype(S)::value;
#pragma unroll
    for (int i = 0; i < TILES; ++i) multiply<FP4, NT>(acc[i], c[s][i], t[s], lane);
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  if (first >= end) return;
  load(S0{}, first);
  for (int chunk = first; chunk < end; chunk += 2 * step) {
    if (chunk + step < end) load(S1{}, chunk + step);
    multiply_all(S0{});
    if (chunk + step >= end) break;
    if (chunk + 2 * step < end) load(S0{}, chunk + 2 * step);
    multiply_all(S1{});
  }
}

template <bool FP4>
__device__ __forceinline__ Matrix expert_matrix(const void* b, const void* sf, int e, int rows, int k) {
  Matrix m;
  m.k = k;
  m.ld = rows;  // a multiple of 128, and so aligned
  const size_t values = (size_t)rows * k;
  m.w = static_cast<const uint8_t*>(b) + (size_t)e * (FP4 ? values / 2 : values);
  m.sf = static_cast<const uint32_t*>(sf) + (size_t)e * (FP4 ? values / QBLOCK : values / QBLOCK / 128);
  return m;
}

// ---------------------------------------------------------------------------
// Up
// ---------------------------------------------------------------------------

constexpr int UP_WAVES = 4, UP_THREADS = UP_WAVES * 64;

// Whether slot i is the first of its token with its expert.
__device__ __forceinline__ bool first_of_token(const int* ids, int i, int top_k) {
  const int e = ids[i];
  for (int j = i - i % top_k; j < i; ++j)
    if (ids[j] == e) return false;
  return true;
}

// The plan, by one workgroup: every slot looks at all others (LDS, all lanes at
// the same one), at most 1024 of them.
__device__ void build_plan(const ExpertsArgs& p, ExpertPlan* plan, const int* ids, int* owner) {
  const int n = p.tokens * p.top_k;
  // owner[i]: the first slot of i's expert, where i is its pair's first slot; else n.
  for (int i = threadIdx.x; i < n; i += UP_THREADS) {
    const int e = ids[i];
    int own = n;
    if (e >= 0 && e < p.num_groups && first_of_token(ids, i, p.top_k)) {
      own = i;
      for (int j = 0; j < i; ++j)
        if (ids[j] == e) {
          own = j;
          break;
        }
    }
    owner[i] = own;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += UP_THREADS) {
    const int own = owner[i];
    if (own == n) continue;
    int at = 0, rank = 0, begin = 0, count = 0;
    for (int j = 0; j < n; ++j) {
      const int other = owner[j];
      at += other < own || (other == own && j < i);
      begin += other < own;
      count += other == own;
      rank += other == j && j < own;
    }
    float w = 0.0f;
    const int t0 = i - i % p.top_k;
    for (int j = t0; j < t0 + p.top_k; ++j)
      if (ids[j] == ids[i]) w += p.weights ? p.weights[j] : 1.0f;
    plan->slot[at] = i;
    plan->weight[at] = w;
    if (own == i) plan->entry[rank] = ExpertEntry{ids[i], begin, count, 0};
  }
  if (threadIdx.x == 0) {
    int experts = 0, pairs = 0;
    for (int j = 0; j < n; ++j) {
      pairs += owner[j] != n;
      experts += owner[j] == j;
    }
    plan->experts = experts;
    plan->pairs = pairs;
  }
}

// One pass of an expert's workgroup over its rows with up to 16 NT tokens: the
// waves share K and their sums meet in LDS.
template <bool FP4, int RT, int NT>
__device__ void up_pass(const ExpertsArgs& p, const Matrix& m, int f0, const int* slots, int count, f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const uint16_t* row[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    row[nt] = p.x + (size_t)(slots[min(nt * 16 + r, count - 1)] / p.top_k) * p.hidden;
  int row0[2 * RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    row0[i] = f0 + 16 * i;
    row0[RT + i] = p.inner + f0 + 16 * i;
  }
  f32x4 acc[2 * RT][NT];
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[i][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int chunks = (m.k / QBLOCK + CHUNK_BLOCKS<FP4> - 1) / CHUNK_BLOCKS<FP4>;
  stream_rows<FP4, 2 * RT, NT>(acc, m, row0, row, wave, UP_WAVES, chunks, lane);

  constexpr int UNITS = 2 * RT * NT;
  __syncthreads();  // of an earlier pass: its sums have been read
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) red[(wave * UNITS + i * NT + nt) * 64 + lane] = acc[i][nt];
  __syncthreads();
  for (int unit = wave; unit < RT * NT; unit += UP_WAVES) {
    f32x4 gate = red[unit * 64 + lane], up = red[(RT * NT + unit) * 64 + lane];
#pragma unroll
    for (int w = 1; w < UP_WAVES; ++w) {
      gate += red[(w * UNITS + unit) * 64 + lane];
      up += red[(w * UNITS + RT * NT + unit) * 64 + lane];
    }
    f32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = gate[i] * sigmoid(gate[i]) * up[i];
    const int i = unit / NT, t = (unit % NT) * 16 + r;
    if (t < count) {
      const u32x2 packed = {pack2((f32x2){a[0], a[1]}), pack2((f32x2){a[2], a[3]})};
      *reinterpret_cast<u32x2*>(p.act + (size_t)slots[t] * p.inner + f0 + 16 * i + 4 * g) = packed;
    }
  }
}

// Workgroup 0 makes the plan; the others take 16 RT gate rows and as many up rows
// of one expert each: an expert by its number, or with more experts than slots the
// expert of a slot that is the first to name it.
template <bool FP4, int RT, int NT>
__global__ __launch_bounds__(UP_THREADS) void experts_up_kernel(ExpertsArgs p) {
  __shared__ int ids[MAX_FEW_PAIRS];
  __shared__ int list[MAX_FEW_PAIRS];  // the plan's owners; else the expert's slots
  __shared__ int waves_before[UP_WAVES + 1];
  __shared__ f32x4 red[UP_WAVES * 2 * RT * NT * 64];
  const int n = p.tokens * p.top_k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < n; i += UP_THREADS) ids[i] = p.ids[i];
  __syncthreads();
  if (blockIdx.x == 0) {
    build_plan(p, reinterpret_cast<ExpertPlan*>(p.plan), ids, list);
    return;
  }
  const int tiles = p.inner / (16 * RT), item = (blockIdx.x - 1) / tiles, f0 = (blockIdx.x - 1) % tiles * 16 * RT;
  const bool by_slot = n <= p.num_groups;
  const int e = by_slot ? ids[item] : item;
  if (e < 0 || e >= p.num_groups) return;
  // The expert's slots in order, counted 256 at a time.
  int count = 0;
  bool earlier = false;
  for (int i0 = 0; i0 < n; i0 += UP_THREADS) {
    const int i = i0 + tid;
    const bool mine = i < n && ids[i] == e;
    const bool take = mine && first_of_token(ids, i, p.top_k);
    earlier |= mine && by_slot && i < item;
    const uint64_t votes = __ballot(take);
    if (lane == 0) waves_before[wave] = __popcll(votes);
    __syncthreads();
    int before = count;
    for (int w = 0; w < UP_WAVES; ++w) {
      if (w < wave) before += waves_before[w];
      count += waves_before[w];
    }
    if (take) list[before + __popcll(votes & ((1ull << lane) - 1))] = i;
    __syncthreads();
  }
  if (__syncthreads_or(earlier) || count == 0) return;

  const Matrix m = expert_matrix<FP4>(p.b1, p.sfb1, e, 2 * p.inner, p.hidden);
  for (int t0 = 0; t0 < count; t0 += 16 * NT) {
    const int here = min(count - t0, 16 * NT);
    if (NT == 1 || here <= 16) up_pass<FP4, RT, 1>(p, m, f0, list + t0, here, red);
    else if (NT == 2 || here <= 32) up_pass<FP4, RT, std::min(NT, 2)>(p, m, f0, list + t0, here, red);
    else up_pass<FP4, RT, NT>(p, m, f0, list + t0, here, red);
  }
}

// ---------------------------------------------------------------------------
// Down
// ---------------------------------------------------------------------------

constexpr int DOWN_WAVES = 8, DOWN_THREADS = DOWN_WAVES * 64;

// A workgroup takes 16 RT columns of y for all tokens. Its waves share the experts
// and, where these do not come out even, each expert's K in parts; each wave keeps
// sums of its own in LDS, which are added in order at the end.
template <bool FP4, int RT, int NT>
__device__ __forceinline__ void down_pass(const ExpertsArgs& p, const Matrix& m, int c0, const int* slots,
                                          const float* weights, int count, int first, int end, float* sums,
                                          int stride) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint16_t* row[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) row[nt] = p.act + (size_t)slots[min(nt * 16 + r, count - 1)] * p.inner;
  int row0[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) row0[i] = c0 + 16 * i;
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[i][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};
  stream_rows<FP4, RT, NT>(acc, m, row0, row, first, 1, end, lane);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int t = nt * 16 + r;
    if (t < count) {  // the tile's tokens differ from one another
      const float w = weights[t];
      float* at = sums + (slots[t] / p.top_k) * stride + 4 * g;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        f32x4 s = *reinterpret_cast<f32x4*>(at + 16 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = __builtin_fmaf(w, acc[i][nt][k], s[k]);
        *reinterpret_cast<f32x4*>(at + 16 * i) = s;
      }
    }
  }
}

template <bool FP4, int RT, int TOKENS>
__global__ __launch_bounds__(DOWN_THREADS) void experts_down_kernel(ExpertsArgs p) {
  constexpr int STRIDE = 16 * RT + 4;  // floats; 4 past a power of two, for the banks
  __shared__ float sums[DOWN_WAVES * TOKENS * STRIDE];
  const ExpertPlan* plan = reinterpret_cast<const ExpertPlan*>(p.plan);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c0 = blockIdx.x * 16 * RT;
  float* mine = sums + wave * TOKENS * STRIDE;
  for (int i = threadIdx.x & 63; i < p.tokens * STRIDE; i += 64) mine[i] = 0.0f;

  const int experts = plan->experts, chunks = (p.inner / QBLOCK + CHUNK_BLOCKS<FP4> - 1) / CHUNK_BLOCKS<FP4>;
  // Parts of an expert's K: so many that the waves have the same number of them, or eight rounds.
  int parts = 1;
  while (parts < DOWN_WAVES && parts * 2 <= chunks && experts * parts % DOWN_WAVES && experts * parts < 8 * DOWN_WAVES)
    parts *= 2;
  for (int item = wave; item < experts * parts; item += DOWN_WAVES) {
    const ExpertEntry entry = plan->entry[item / parts];
    const int part = item % parts, first = chunks * part / parts, end = chunks * (part + 1) / parts;
    const Matrix m = expert_matrix<FP4>(p.b2, p.sfb2, entry.expert, p.hidden, p.inner);
    for (int t0 = 0; t0 < entry.count; t0 += 64) {
      const int here = min(entry.count - t0, 64);
      const int* slots = plan->slot + entry.begin + t0;
      const float* weights = plan->weight + entry.begin + t0;
      if (TOKENS <= 16 || here <= 16) down_pass<FP4, RT, 1>(p, m, c0, slots, weights, here, first, end, mine, STRIDE);
      else if (here <= 32) down_pass<FP4, RT, 2>(p, m, c0, slots, weights, here, first, end, mine, STRIDE);
      else down_pass<FP4, RT, 4>(p, m, c0, slots, weights, here, first, end, mine, STRIDE);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.tokens * 8 * RT; i += DOWN_THREADS) {
    const int t = i / (8 * RT), c = i % (8 * RT) * 2;
    f32x2 s = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < DOWN_WAVES; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) s[k] += sums[(w * TOKENS + t) * STRIDE + c + k];
    *reinterpret_cast<uint32_t*>(p.y + (size_t)t * p.hidden + c0 + c) = pack2(s);
  }
}

template <bool FP4, int RT>
hipError_t launch_typed(const ExpertsArgs& a, hipStream_t stream) {
  const int n = a.tokens * a.top_k;
  const int ups = 1 + std::min(n, a.num_groups) * (a.inner / (16 * RT));
  auto* up = a.tokens <= 16 ? experts_up_kernel<FP4, RT, 1>
                            : a.tokens <= 32 ? experts_up_kernel<FP4, RT, 2> : experts_up_kernel<FP4, RT, 4>;
  hipLaunchKernelGGL(up, dim3(ups), dim3(UP_THREADS), 0, stream, a);
  if (hipError_t e = hipGetLastError()) return e;
  auto* down = a.tokens <= 16 ? experts_down_kernel<FP4, RT, 16>
                              : a.tokens <= 64 ? experts_down_kernel<FP4, RT, 64>
                                               : experts_down_kernel<FP4, RT, MAX_FEW_TOKENS>;
  hipLaunchKernelGGL(down, dim3(a.hidden / (16 * RT)), dim3(DOWN_THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts(const ExpertsArgs& a, hipStream_t stream) {
  return a.fp4 ? launch_typed<true, 1>(a, stream) : launch_typed<false, 1>(a, stream);
}

}  // namespace moe
}  // namespace dg
