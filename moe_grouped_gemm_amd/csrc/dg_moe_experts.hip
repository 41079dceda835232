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
// the lane is weight row 4g + i for token r. Lane group g takes a quarter of a
// 128-value block in four such instructions: of FP4 K positions 32g .. 32g + 31, one
// scale's; of FP8 16g .. 16g + 15 and 64 more, so that the four groups' loads are 64
// bytes of a row in either case. (Which positions those are is free, as long as the
// tokens' values are the same ones.)
//
// The weights are read by plain loads: half a line at a time of 16 rows, streaming
// ones reach 5.6 TB/s in a kernel that only reads, plain ones 6.3 (long rows read
// through 6.8, 6.2).

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

// One expert's matrix [rows][k] and its scales.
struct Matrix {
  const uint8_t* w;
  const uint32_t* sf;  // FP8: floats [rows/128][k/128]; FP4: words [k/128][rows]
};

// What is the same for every expert and step: sizes, and the lane's places.
template <bool FP4>
struct Shape {
  int rows, k;
  size_t row_bytes;
  uint32_t w_at, sf_at;  // of lane (r, g) in a tile's block: bytes; words

  __device__ Shape(int rows_, int k_, int lane)
      : rows(rows_), k(k_), row_bytes(FP4 ? k_ / 2 : k_),
        w_at((uint32_t)(lane & 15) * (uint32_t)row_bytes + (lane >> 4) * 16), sf_at(FP4 ? lane & 15 : 0) {}
  __device__ Matrix expert(const void* b, const void* sf, int e) const {
    const size_t values = (size_t)rows * k;
    return Matrix{static_cast<const uint8_t*>(b) + (size_t)e * (FP4 ? values / 2 : values),
                  static_cast<const uint32_t*>(sf) + (size_t)e * (FP4 ? values / QBLOCK : values / QBLOCK / 128)};
  }
};

// One 128-value block of a 16-row tile as loaded: lane (r, g) of row r.
template <bool FP4>
struct Tile {
  u32x4 w[FP4 ? 1 : 2];  // bytes 16g .. 16g + 15 and, FP8, 64 + 16g .. + 15
  uint32_t sf;
};

template <bool FP4>
__device__ __forceinline__ void load_tile(Tile<FP4>& t, const Shape<FP4>& sh, const Matrix& m, int row0, int block) {
  const uint8_t* src = m.w + (size_t)row0 * sh.row_bytes + (size_t)block * (FP4 ? 64 : 128);
  t.w[0] = load16(src + sh.w_at);
  if constexpr (!FP4) t.w[1] = load16(src + sh.w_at + 64);
  const uint32_t* sf = FP4 ? m.sf + (size_t)block * sh.rows + row0 : m.sf + (size_t)(row0 / 128) * (sh.k / QBLOCK) + block;
  t.sf = sf[sh.sf_at];
}

__device__ __forceinline__ bf16x8 as_operand(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// The four operands of the block.
template <bool FP4>
__device__ __forceinline__ void operands(const Tile<FP4>& t, int g, bf16x8 (&out)[4]) {
  if constexpr (FP4) {
    const uint32_t code = (t.sf >> (8 * g)) & 0xFF;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t dword = t.w[0][j];
      out[j] = as_operand(fp4_values(dword, code));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = t.w[j / 2][2 * (j & 1)], hi = t.w[j / 2][2 * (j & 1) + 1];
      const u32x4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
      out[j] = as_operand(v);
    }
  }
}

// A step: one 128-value block of K of TILES 16-row tiles and of 16 NT tokens, lane
// (r, g) of row or token r.
template <bool FP4, int TILES, int NT>
struct Step {
  Tile<FP4> w[TILES];
  u32x4 t[NT][4];
};

template <bool FP4, int NT>
__device__ __forceinline__ void load_tokens(u32x4 (&t)[NT][4], const uint16_t* const (&row)[NT], int block, int lane) {
  const int g = lane >> 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      t[nt][j] = load16(row[nt] + block * QBLOCK + (FP4 ? 32 * g + 8 * j : 64 * (j >> 1) + 16 * g + 8 * (j & 1)));
}

template <bool FP4, int TILES, int NT>
__device__ __forceinline__ void multiply(f32x4 (&acc)[TILES][NT], const Step<FP4, TILES, NT>& s, int lane) {
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    bf16x8 w[4];
    operands<FP4>(s.w[i], lane >> 4, w);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (FP4) {  // the scales are in the operands
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], as_operand(s.t[nt][j]), acc[i][nt], 0, 0, 0);
      } else {
        const float scale = __builtin_bit_cast(float, s.w[i].sf);
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], as_operand(s.t[nt][j]), part, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][nt][k] = __builtin_fmaf(part[k], scale, acc[i][nt][k]);
      }
    }
  }
}

// Runs steps 0 .. n-1 with DEPTH of them in registers: load(buffer, i) is called
// DEPTH - 1 steps ahead of use(buffer, i), in order, without a condition around it
// (past the last step it is asked for the last one again), in rounds that are left
// at their end only: on every path to a use the compiler then knows how many loads
// follow the ones that it waits for.
template <int DEPTH, class BUFFER, class LOAD, class USE>
__device__ __forceinline__ void pipeline(int n, LOAD&& load, USE&& use) {
  BUFFER buf[DEPTH];
  if (n <= 0) return;
  static_for<0, DEPTH - 1>([&](auto I) { load(buf[decltype(I)::value], min((int)decltype(I)::value, n - 1)); });
  const int rounds = n / DEPTH * DEPTH;
  for (int i0 = 0; i0 < rounds; i0 += DEPTH) {
    static_for<0, DEPTH>([&](auto I) {
      constexpr int j = decltype(I)::value;
      load(buf[(j + DEPTH - 1) % DEPTH], min(i0 + j + DEPTH - 1, n - 1));
      use(buf[j], i0 + j);
    });
  }
  static_for<0, DEPTH - 1>([&](auto I) {
    constexpr int j = decltype(I)::value;
    if (rounds + j < n) use(buf[j], rounds + j);
  });
}

// ---------------------------------------------------------------------------
// Up
// ---------------------------------------------------------------------------

constexpr int UP_WAVES = 4, UP_THREADS = UP_WAVES * 64;

// The i-th block of K that a wave takes, and how many there are: turn by turn, for
// FP4 two successive ones, which share a 128-byte line of a row.
template <bool FP4>
__device__ __forceinline__ int wave_block(int wave, int i) {
  return FP4 ? (i >> 1) * 2 * UP_WAVES + 2 * wave + (i & 1) : i * UP_WAVES + wave;
}
template <bool FP4>
__device__ __forceinline__ int wave_blocks(int wave, int blocks) {
  if (!FP4) return (blocks - wave + UP_WAVES - 1) / UP_WAVES;
  const int rounds = blocks / (2 * UP_WAVES);
  return 2 * rounds + min(max(blocks - rounds * 2 * UP_WAVES - 2 * wave, 0), 2);
}

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

// Steps in registers.
template <bool FP4, int NT>
constexpr int UP_DEPTH = FP4 && NT == 1 ? 3 : 2;

// One pass of an expert's workgroup over its rows with up to 16 NT tokens: the
// waves share K and their sums meet in LDS.
template <bool FP4, int RT, int NT>
__device__ __forceinline__ void up_pass(const ExpertsArgs& p, const Shape<FP4>& shape, const Matrix& m, int f0,
                                        const int* slots, int count, f32x4* red) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
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
  using Buffer = Step<FP4, 2 * RT, NT>;
  pipeline<UP_DEPTH<FP4, NT>, Buffer>(
      wave_blocks<FP4>(wave, p.hidden / QBLOCK),
      [&](Buffer& s, int i) {
        const int block = wave_block<FP4>(wave, i);
#pragma unroll
        for (int k = 0; k < 2 * RT; ++k) load_tile<FP4>(s.w[k], shape, m, row0[k], block);
        load_tokens<FP4, NT>(s.t, row, block, lane);
      },
      [&](const Buffer& s, int) { multiply<FP4, 2 * RT, NT>(acc, s, lane); });

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

  const Shape<FP4> shape(2 * p.inner, p.hidden, lane);
  const Matrix m = shape.expert(p.b1, p.sfb1, __builtin_amdgcn_readfirstlane(e));
  for (int t0 = 0; t0 < count; t0 += 16 * NT) {
    const int here = min(count - t0, 16 * NT);
    if (NT == 1 || here <= 16) up_pass<FP4, RT, 1>(p, shape, m, f0, list + t0, here, red);
    else up_pass<FP4, RT, NT>(p, shape, m, f0, list + t0, here, red);
  }
}

// ---------------------------------------------------------------------------
// Down
// ---------------------------------------------------------------------------

constexpr int DOWN_WAVES = 8, DOWN_THREADS = DOWN_WAVES * 64;

// A workgroup takes 16 RT columns of y for all tokens. Its waves share the experts,
// 16 tokens of one at a time, and, where these do not come out even, their K in
// parts; each wave keeps sums of its own in LDS, which are added in order at the end.
// A wave's items follow one another in one pipeline of steps.
template <bool FP4>
constexpr int DOWN_DEPTH = FP4 ? 4 : 3;

struct DownItem {
  int expert, begin, count;  // pairs of the plan, at most 16
};

template <bool FP4, int RT, int TOKENS>
__global__ __launch_bounds__(DOWN_THREADS) void experts_down_kernel(ExpertsArgs p) {
  constexpr int STRIDE = 16 * RT + (TOKENS > 64 ? 0 : 4);  // floats; 4 past a power of two where there is room
  __shared__ float sums[DOWN_WAVES * TOKENS * STRIDE];
  __shared__ DownItem items[MAX_FEW_PAIRS];
  __shared__ int items_of[DOWN_THREADS / 64];
  // Of the pairs; read from memory in the loop, they would be waited for with all the
  // weights that are on their way.
  __shared__ int slots[MAX_FEW_PAIRS];
  __shared__ uint16_t sums_at[MAX_FEW_PAIRS];  // of the pair's token, in 16 bytes
  __shared__ float weights[MAX_FEW_PAIRS];
  const ExpertPlan* plan = reinterpret_cast<const ExpertPlan*>(p.plan);
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), c0 = blockIdx.x * 16 * RT;
  float* mine = sums + wave * TOKENS * STRIDE;
  for (int i = lane; i < p.tokens * STRIDE; i += 64) mine[i] = 0.0f;

  const int experts = plan->experts, pairs = plan->pairs;
  for (int i = tid; i < pairs; i += DOWN_THREADS) {
    const int slot = plan->slot[i];
    slots[i] = slot;
    sums_at[i] = (uint16_t)(slot / p.top_k * (STRIDE / 4));
    weights[i] = plan->weight[i];
  }
  // The items: an expert's pairs 16 at a time, in order.
  int total = 0;
  for (int r0 = 0; r0 < experts; r0 += DOWN_THREADS) {
    const int at = r0 + tid;
    ExpertEntry entry{0, 0, 0, 0};
    if (at < experts) entry = plan->entry[at];
    const int has = (entry.count + 15) / 16;
    int upto = has;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) items_of[wave] = upto;
    __syncthreads();
    int before = total + upto - has;
    for (int w = 0; w < DOWN_THREADS / 64; ++w) {
      if (w < wave) before += items_of[w];
      total += items_of[w];
    }
    for (int i = 0; i < has; ++i)
      items[before + i] = DownItem{entry.expert, entry.begin + 16 * i, min(entry.count - 16 * i, 16)};
    __syncthreads();
  }

  // Parts of K (of pairs of blocks, see wave_block): so many that the waves have the
  // same number of items, or that they have eight each.
  const int blocks = p.inner / QBLOCK, unit = FP4 ? 2 : 1, units = (blocks + unit - 1) / unit;
  int parts = 1;
  while (parts < DOWN_WAVES && parts * 2 <= units && total * parts % DOWN_WAVES && total * parts < 8 * DOWN_WAVES)
    parts *= 2;
  const int all = total * parts, turns = wave < all ? (all - wave + DOWN_WAVES - 1) / DOWN_WAVES : 0;

  const Shape<FP4> shape(p.hidden, p.inner, lane);
  // Where the loads and the products are: the turn, its item and its blocks.
  struct Cursor {
    int turn, block, end, begin, count;
    Matrix m;
  };
  auto start = [&](Cursor& c) {
    const int item = wave + c.turn * DOWN_WAVES, part = item % parts;
    const DownItem at = items[item / parts];
    c.begin = __builtin_amdgcn_readfirstlane(at.begin);
    c.count = __builtin_amdgcn_readfirstlane(at.count);
    c.m = shape.expert(p.b2, p.sfb2, __builtin_amdgcn_readfirstlane(at.expert));
    c.block = units * part / parts * unit;
    c.end = min(units * (part + 1) / parts * unit, blocks);
  };
  int steps = 0;
  for (int turn = 0; turn < turns; ++turn) {
    const int part = (wave + turn * DOWN_WAVES) % parts;
    steps += min(units * (part + 1) / parts * unit, blocks) - units * part / parts * unit;
  }

  using Buffer = Step<FP4, RT, 1>;
  Cursor ahead{}, now{};
  const uint16_t* row[1] = {p.act};
  f32x4 acc[RT][1] = {};
  int loaded = 0;
  if (steps > 0) {
    start(ahead);
    start(now);
    row[0] = p.act + (size_t)slots[ahead.begin + min(r, ahead.count - 1)] * p.inner;
  }
  pipeline<DOWN_DEPTH<FP4>, Buffer>(
      steps,
      [&](Buffer& s, int) {
#pragma unroll
        for (int i = 0; i < RT; ++i) load_tile<FP4>(s.w[i], shape, ahead.m, c0 + 16 * i, ahead.block);
        load_tokens<FP4, 1>(s.t, row, ahead.block, lane);
        if (++loaded < steps && ++ahead.block == ahead.end) {
          ++ahead.turn;
          start(ahead);
          row[0] = p.act + (size_t)slots[ahead.begin + min(r, ahead.count - 1)] * p.inner;
        }
      },
      [&](const Buffer& s, int i) {
        multiply<FP4, RT, 1>(acc, s, lane);
        if (++now.block < now.end) return;
        if (r < now.count) {  // the item's tokens differ from one another
          const float w = weights[now.begin + r];
          float* at = mine + 4 * (sums_at[now.begin + r] + g);
#pragma unroll
          for (int k = 0; k < RT; ++k) {
            f32x4 sum = *reinterpret_cast<f32x4*>(at + 16 * k);
#pragma unroll
            for (int v = 0; v < 4; ++v) sum[v] = __builtin_fmaf(w, acc[k][0][v], sum[v]);
            *reinterpret_cast<f32x4*>(at + 16 * k) = sum;
          }
        }
#pragma unroll
        for (int k = 0; k < RT; ++k) acc[k][0] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (i + 1 < steps) {
          ++now.turn;
          start(now);
        }
      });
  __syncthreads();
  for (int i = tid; i < p.tokens * 8 * RT; i += DOWN_THREADS) {
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
  auto* up = a.tokens <= 16 ? experts_up_kernel<FP4, RT, 1> : experts_up_kernel<FP4, RT, 2>;
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
  return a.fp4 ? launch_typed<true, 2>(a, stream) : launch_typed<false, 2>(a, stream);
}

}  // namespace moe
}  // namespace dg
