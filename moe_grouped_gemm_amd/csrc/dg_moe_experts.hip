// A whole expert layer for a few tokens in two launches:
//
//   a[t, e] = silu(g) * u,  [g | u] = B1[e] x[t]             (up)
//   y[t]    = sum_j w[t, j] * B2[e] a[t, e], e = ids[t, j]   (down)
//
// with the experts' weights in FP8 (one float32 scale per 128 x 128) or FP4 (one
// power-of-two scale per 32 values of a row) and everything else as it comes: x in
// BF16, sums in float32, a held to 2^-16 of it in two BF16 values, y rounded once. The
// weights of an expert are read once for each 32 of its tokens, and that bounds both
// launches.
//
// Every wave streams weights of its own through a ring in LDS, without a barrier:
// direct-to-LDS loads whose successive lanes read a row's successive 16 bytes, some
// steps ahead; each step it waits for its own oldest ones, reads them as the matrix
// cores want them, converts them to BF16 (exact: E4M3 has 4 significant bits, E2M1 2)
// and multiplies them with up to 16 tokens a tile. Loads straight into the matrix
// cores' registers, lane by lane a row, take the L1 four times the accesses: one
// 16-byte piece each, 3.4 TB/s where tokens' rows come the same way.
//
// What bounds it: a compute unit takes some 40 GB/s together, whether two or five
// steps are on their way, so the tokens' or activations' bytes (16 tokens: half the
// weights' in the first launch, twice as many in the second) and the processors' turns
// add to the weights' time. An FP8 batch, 61 tokens and 32 experts of 7168 x 2048:
// 183 us (5.1 TB/s of weights) and 129 (3.7); weights alone 164 and 79, and the second
// launch 102 with activations of one BF16 value. One token, eight experts in FP4: 28 and 18
// us, of which about 5 each are a launch's lists of who is where, one read from memory
// after the other.
//
// A step is 128 bytes of each row: 128 values of FP8, or two blocks of 128 of FP4.
//
// v_mfma_f32_16x16x32_bf16: the first operand's lane (r, g) = (lane % 16, lane /
// 16) holds 8 values of K of weight row r, the second's of token r, and result i of
// the lane is weight row 4g + i for token r. Lane group g takes a quarter of a
// 128-value block in four such instructions j: of FP4 K positions 32g + 8j .. + 7,
// one scale's; of FP8 64 (j / 2) + 16g + 8 (j % 2) .. + 7, which are 16-byte pieces g
// and g + 4 of the row. (Which positions those are is free, as long as the tokens'
// values are the same ones.)

#include <algorithm>

#include "dg_device.h"
#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

// Columns that the second launch spreads over the chip, 16 to a compute unit: with fewer
// columns of y, several workgroups share the experts of 16 columns.
constexpr int DOWN_COLUMNS = EXPERT_DOWN_COLUMNS;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What the first launch leaves for the second, before the activations: the experts
// that have tokens, in order of their first slot, and their (token, expert) pairs.
// A pair is known by its first slot; a token that names an expert twice is one pair
// with the weights' sum.
struct ExpertEntry {
  int expert, begin, count, first;  // its pairs, and the slot of the first
};
struct ExpertPlan {
  int experts, pad[3];
  ExpertEntry entry[MAX_FEW_PAIRS];
  int slot[MAX_FEW_PAIRS];
  float weight[MAX_FEW_PAIRS];
  int done[DOWN_COLUMNS / 16];  // of each 16 columns of y: workgroups whose sums are there
};
static_assert(sizeof(ExpertPlan) == EXPERT_PLAN_BYTES, "room for the plan");

// ---------------------------------------------------------------------------
// Activations between the launches
// ---------------------------------------------------------------------------

// A value is held as the sum of two in BF16, float32's upper 16 bits and what those leave
// out, which is good to 2^-16 of it (with one BF16 value, good to 2^-8, the layer's error
// was 0.0023 in the 2-norm, where y's own rounding makes 0.0017). The second products multiply the two side by side, as neighbouring
// columns of a token operand: a tile is one expert's up to 8 tokens.
//
// Tiles lie in the order in which the second launch's lanes load them, 16 bytes each: block
// b of 128 values, instruction j, lane group g, row: each token's upper part, then its
// lower one, so that few tokens take few cache lines (with all upper parts first, 16 tokens
// and 64 experts took 88 us for 69). TOKENS, of a tile, is 4 where the call has no more,
// else 8. With no more slots than experts a tile is known by its first pair's slot, else by
// the expert and its number.
constexpr int TILE_TOKENS = 8;
__device__ __forceinline__ bool tiles_by_slot(const ExpertsArgs& p) { return p.tokens * p.top_k <= p.num_groups; }
__device__ __forceinline__ int act_tile(const ExpertsArgs& p, int expert, int number, int first_slot) {
  return tiles_by_slot(p) ? first_slot : expert * ((p.tokens + TILE_TOKENS - 1) / TILE_TOKENS) + number;
}
// Of value k of a tile's row, in BF16 values.
template <bool FP4, int TOKENS>
__device__ __forceinline__ int act_at(int k, int row) {
  const int b = k / QBLOCK, in = k % QBLOCK;
  const int g = FP4 ? in / 32 : in / 16 % 4, j = FP4 ? in / 8 % 4 : in / 64 * 2 + in / 8 % 2;
  return b * QBLOCK * 2 * TOKENS + ((j * 4 + g) * 2 * TOKENS + row) * 8 + in % 8;
}

// The upper parts of two values, and the lower ones (nothing is left of an infinity).
__device__ __forceinline__ uint32_t upper2(float a, float b) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
}
__device__ __forceinline__ uint32_t lower2(float a, float b) {
  auto rest = [](float v) {
    return __builtin_isfinite(v) ? v - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u) : 0.0f;
  };
  return pack2((f32x2){rest(a), rest(b)});
}

// ---------------------------------------------------------------------------
// Weights
// ---------------------------------------------------------------------------

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds), 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds), 4, voff, soff, 0, 0);
}

// Neither the loads' waits nor their LDS writes are seen by the compiler: no access to
// LDS moves past these.
template <int N>
__device__ __forceinline__ void wait_loads() {
  wait_vmcnt<N>();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void before_loads() {
  wait_lgkmcnt_0();  // what a slot held has been read
  asm volatile("" ::: "memory");
}

// One step of the weights: 128 bytes of each row of TILES 16-row tiles, GROUPS (1 or 2)
// runs of successive rows, with their scales.
template <bool FP4, int TILES_, int GROUPS>
struct Weights {
  static constexpr int TILES = TILES_, PER_GROUP = TILES / GROUPS;
  static constexpr int BLOCKS = FP4 ? 2 : 1;  // of 128 values, in a step
  static constexpr int TILE_BYTES = 2048, SCALES_AT = TILES * TILE_BYTES;
  static constexpr int SCALE_LOADS = FP4 ? (TILES + 1) / 2 : 1;
  static constexpr int BYTES = SCALES_AT + SCALE_LOADS * 256;  // of a step in LDS
  static constexpr int LOADS = TILES * 2 + SCALE_LOADS;

  const uint8_t* b;
  const uint32_t* sf;
  int n, k;                                      // the matrix is [n][k]
  uint32_t row_bytes, scale_step;                // bytes between rows; between a step's scales and the next's
  uint32_t w_at[2];                              // the lane's offsets,
  uint32_t read_at, read_sf;                     // and in LDS
  __amdgpu_buffer_rsrc_t rows[GROUPS], scales;   // of the place at hand
  uint32_t sf_at[SCALE_LOADS];

  __device__ __forceinline__ Weights(const void* b_, const void* sf_, int n_, int k_, int lane)
      : b(static_cast<const uint8_t*>(b_)), sf(static_cast<const uint32_t*>(sf_)), n(n_), k(k_) {
    const int r = lane & 15, g = lane >> 4;
    row_bytes = FP4 ? k / 2 : k;
    scale_step = FP4 ? n * 8 : 4;
    // A load is 8 rows of 128 bytes; pieces of 16 are swizzled for the fragment reads.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * h + (lane >> 3), piece = (lane & 7) ^ ((row >> 1) & 7);
      w_at[h] = row * row_bytes + piece * 16;
    }
    read_at = lds_offset(r, g);  // and, with bit 6 flipped, lds_offset(r, g + 4)
    read_sf = r * 4;
  }

  // Turns to the runs of rows from row0[.] of expert e's matrix.
  __device__ __forceinline__ void place(int e, const int (&row0)[GROUPS], int lane) {
    // What lies past the expert's matrix (a last block of FP4 may have no second one) reads
    // as zero.
    const size_t values = (size_t)n * k, bytes = FP4 ? values / 2 : values;
    const size_t sf_words = FP4 ? values / QBLOCK : values / QBLOCK / 128;
    auto extent = [](size_t left) { return (uint32_t)min(left, (size_t)0xFFFFFFFFu); };
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const size_t at = (size_t)row0[i] * row_bytes;
      rows[i] = buffer_rsrc(b + e * bytes + at, extent(bytes - at));
    }
    scales = buffer_rsrc(sf + e * sf_words, extent(sf_words * 4));
    // (By value: a choice between the array's elements would put it in memory.)
    const int run0 = row0[0], run1 = row0[GROUPS - 1];
    if constexpr (FP4) {
      // Words of the first block's rows, then the second's.
#pragma unroll
      for (int q = 0; q < SCALE_LOADS; ++q) {
        const int at = min(4 * q + (lane >> 4), 2 * TILES - 1), block = at / TILES, tile = at % TILES;
        const int group = tile / PER_GROUP;
        sf_at[q] = (block * n + (group ? run1 : run0) + (tile - group * PER_GROUP) * 16 + (lane & 15)) * 4;
      }
    } else {
      sf_at[0] = (lane & 1 ? run1 : run0) / 128 * (k / QBLOCK) * 4;
    }
  }

  __device__ __forceinline__ void load(int step, uint32_t lds) const {
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        dma16(rows[i / PER_GROUP], w_at[h], (uint32_t)(i % PER_GROUP) * 16 * row_bytes + (uint32_t)step * 128,
              lds + i * TILE_BYTES + h * 1024);
#pragma unroll
    for (int q = 0; q < SCALE_LOADS; ++q) dma4(scales, sf_at[q], (uint32_t)step * scale_step, lds + SCALES_AT + q * 256);
  }

  // acc += tile i of block `block` of the step at `st` times the first USED of the tokens'
  // operands.
  template <int USED, int NT>
  __device__ __forceinline__ void multiply(f32x4 (&acc)[NT], const uint8_t* st, int i, int block,
                                           const u32x4 (&t)[NT][4], int lane) const {
    const uint8_t* tile = st + i * TILE_BYTES;
    const uint8_t* sf = st + SCALES_AT;
    bf16x8 w[4];
    if constexpr (FP4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(tile + (block ? read_at ^ 64 : read_at));
      const uint32_t word = *reinterpret_cast<const uint32_t*>(sf + (block * TILES + i) * 64 + read_sf);
      const uint32_t code = (word >> (8 * (lane >> 4))) & 0xFF;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t dword = v[j];
        w[j] = __builtin_bit_cast(bf16x8, fp4_values(dword, code));
      }
#pragma unroll
      for (int nt = 0; nt < USED; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], __builtin_bit_cast(bf16x8, t[nt][j]), acc[nt], 0, 0, 0);
    } else {
      const u32x4 v[2] = {*reinterpret_cast<const u32x4*>(tile + read_at),
                          *reinterpret_cast<const u32x4*>(tile + (read_at ^ 64))};
      const float scale = *reinterpret_cast<const float*>(sf + i / PER_GROUP * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = v[j / 2][2 * (j & 1)], hi = v[j / 2][2 * (j & 1) + 1];
        const u32x4 o = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
        w[j] = __builtin_bit_cast(bf16x8, o);
      }
#pragma unroll
      for (int nt = 0; nt < USED; ++nt) {
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j], __builtin_bit_cast(bf16x8, t[nt][j]), part, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][k] = __builtin_fmaf(part[k], scale, acc[nt][k]);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Up
// ---------------------------------------------------------------------------

constexpr int UP_WAVES = 4, UP_THREADS = UP_WAVES * 64;
constexpr int UP_W_SLOTS = 2;      // steps of weights in a wave's ring: one is on its way, one in use
constexpr int UP_T_BYTES = 16384;  // and bytes of tokens: two steps of 24 or 32, three of up to 16
constexpr int UP_MOST_FOURS = 8;   // most tokens of a pass, in fours

// Tokens' rows of a block come in loads of 4 rows of 256 bytes; their 16-byte pieces
// are swizzled for the fragment reads, as the weights' are.
__device__ __forceinline__ int token_swizzle(int row) { return (row & 3) | ((-(row >> 2) & 3) << 2); }

template <bool FP4, int RT>
using UpWeights = Weights<FP4, 2 * RT, 2>;
template <bool FP4, int RT>
constexpr int UP_RING = UP_W_SLOTS * UpWeights<FP4, RT>::BYTES + UP_T_BYTES;

// A barrier that leaves loads on their way: LDS accesses before it are done after it.
__device__ __forceinline__ void meet() {
  wait_lgkmcnt_0();
  barrier();
}

// Who is where, in LDS.
struct UpLists {
  short ids[MAX_FEW_PAIRS];        // each slot's expert, -1: none
  uint16_t active[MAX_FEW_PAIRS];  // the experts that have slots, in order of their first ones
  uint16_t list[MAX_FEW_PAIRS];    // the pairs of the expert at hand (and of the plan on its way)
  int waves_before[UP_WAVES];
};

// Whether slot i is the first of its token with its expert.
__device__ __forceinline__ bool first_of_token(const short* ids, int i, int top_k) {
  const int e = ids[i];
  for (int j = i - i % top_k; j < i; ++j)
    if (ids[j] == e) return false;
  return true;
}

// Calls put(i, place) for the slots with take(i), in order; returns their number. By the
// whole workgroup.
template <class TAKE, class PUT>
__device__ __forceinline__ int gather(UpLists& l, int n, TAKE&& take, PUT&& put) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int count = 0;
  for (int i0 = 0; i0 < n; i0 += UP_THREADS) {
    const bool mine = i0 + tid < n && take(i0 + tid);
    const uint64_t votes = __ballot(mine);
    if (lane == 0) l.waves_before[wave] = __popcll(votes);
    meet();
    int before = count;
    for (int w = 0; w < UP_WAVES; ++w) {
      if (w < wave) before += l.waves_before[w];
      count += l.waves_before[w];
    }
    if (mine) put(i0 + tid, before + __popcll(votes & ((1ull << lane) - 1)));
    meet();
  }
  return __builtin_amdgcn_readfirstlane(count);
}

// Writes the plan, by one wave: `order` takes each expert's place among the active ones,
// `next` counts its pairs, both of num_groups ints.
__device__ void write_plan(const ExpertsArgs& p, const UpLists& l, int experts, int* order, int* next) {
  ExpertPlan* const plan = reinterpret_cast<ExpertPlan*>(p.plan);
  const int n = p.tokens * p.top_k, lane = threadIdx.x;
  for (int r = lane; r < experts; r += 64) {
    order[l.active[r]] = r;
    next[l.active[r]] = 0;
  }
  wait_lgkmcnt_0();
  // Each expert's pairs, counted; then where they begin.
  const int bits = 32 - __builtin_clz(p.num_groups);
  auto for_pairs = [&](auto&& f) {
    for (int i0 = 0; i0 < n; i0 += 64) {
      const int i = i0 + lane, e = i < n ? l.ids[i] : -1;
      const bool pair = e >= 0 && first_of_token(l.ids, i, p.top_k);
      uint64_t peers = __ballot(pair);
      for (int b = 0; b < bits; ++b) {
        const uint64_t ones = __ballot((e >> b) & 1);
        peers &= ((e >> b) & 1) ? ones : ~ones;
      }
      const int before = pair ? next[e] : 0, rank = __popcll(peers & ((1ull << lane) - 1));
      wait_lgkmcnt_0();
      if (pair && rank == 0) next[e] = before + __popcll(peers);
      wait_lgkmcnt_0();
      if (pair) f(i, e, before + rank);
    }
  };
  for_pairs([&](int i, int e, int at) {
    if (at == 0) plan->entry[order[e]].first = i;
  });
  int pairs = 0;
  for (int r0 = 0; r0 < experts; r0 += 64) {
    const int r = r0 + lane, e = r < experts ? l.active[r] : 0, has = r < experts ? next[e] : 0;
    int upto = has;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (r < experts) {
      plan->entry[r].expert = e;
      plan->entry[r].begin = pairs + upto - has;
      plan->entry[r].count = has;
      next[e] = pairs + upto - has;
    }
    pairs += __shfl(upto, 63);
  }
  wait_lgkmcnt_0();
  for_pairs([&](int i, int e, int at) {
    float w = 0.0f;
    const int t0 = i - i % p.top_k;
    for (int j = t0; j < t0 + p.top_k; ++j)
      if (l.ids[j] == e) w += p.weights ? p.weights[j] : 1.0f;
    plan->slot[at] = i;
    plan->weight[at] = w;
  });
  for (int i = lane; i < DOWN_COLUMNS / 16; i += 64) plan->done[i] = 0;
  if (lane == 0) plan->experts = experts;
}

// The tiles [tile, tile_end) of 16 RT gate rows and as many up rows of one expert, with up
// to 4 FOURS of its tokens: the waves share K and their sums meet in LDS at a tile's end.
// The weights go on from one tile to the next; tokens' rows are fetched again, from L2.
template <bool FP4, int RT, int FOURS, int TOKENS>
__device__ __forceinline__ void up_tiles(const ExpertsArgs& p, UpWeights<FP4, RT>& weights, int tile, int tile_end,
                                         int expert, int number, const uint16_t* slots, int count, uint8_t* lds) {
  constexpr int NT = (FOURS + 3) / 4, W = UpWeights<FP4, RT>::LOADS, T = FOURS, TILES = 2 * RT;
  constexpr int STEP = UpWeights<FP4, RT>::BYTES, TOKEN_BYTES = FOURS * 1024;
  constexpr int T_AHEAD = FOURS <= 4 ? 2 : 1, T_SLOTS = T_AHEAD + 1;
  // The waves' sums lie at the end of their tokens' place; before them the next tile's
  // first tokens are on their way meanwhile.
  constexpr int SUMS = TILES * NT * 1024, SUMS_AT = UP_W_SLOTS * STEP + UP_T_BYTES - SUMS;
  static_assert(T_SLOTS * TOKEN_BYTES <= UP_T_BYTES && T_AHEAD * TOKEN_BYTES + SUMS <= UP_T_BYTES, "room for both");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  uint8_t* const ring = lds + wave * UP_RING<FP4, RT>;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void*)ring, token_base = base + UP_W_SLOTS * STEP;
  const __amdgpu_buffer_rsrc_t x = buffer_rsrc(p.x, 0xFFFFFFFFu);
  constexpr int BLOCKS = UpWeights<FP4, RT>::BLOCKS;
  // Steps of K go to the waves turn by turn: the wave's i-th, of which the last of all may
  // have one block only.
  const int all_blocks = p.hidden / QBLOCK, all_steps = (all_blocks + BLOCKS - 1) / BLOCKS;
  const int steps = max((all_steps - wave + UP_WAVES - 1) / UP_WAVES, 0);
  auto step_of = [&](int i) { return i * UP_WAVES + wave; };
  const int blocks = steps * BLOCKS - (steps > 0 && (step_of(steps - 1) + 1) * BLOCKS > all_blocks);

  // The weights' loads: where they are, a step ahead of the products.
  int w_tile = tile, w_i = 0, w_next = 0;
  auto place = [&]() {
    const int row0[2] = {w_tile * 16 * RT, p.inner + w_tile * 16 * RT};
    weights.place(expert, row0, lane);
  };
  auto load_weights = [&]() {  // (past the last step it is loaded again)
    weights.load(step_of(w_i), base + w_next * STEP);
    w_next = w_next == UP_W_SLOTS - 1 ? 0 : w_next + 1;
    if (w_i + 1 < steps) {
      ++w_i;
    } else if (w_tile + 1 < tile_end) {
      ++w_tile;
      w_i = 0;
      place();
    }
  };
  place();
  if (steps > 0) load_weights();

  uint32_t x_at[FOURS];
#pragma unroll
  for (int q = 0; q < FOURS; ++q) {
    const int row = 4 * q + g;
    x_at[q] = (uint32_t)(slots[min(row, count - 1)] / p.top_k) * (uint32_t)(p.hidden * 2) +
              (uint32_t)((r ^ token_swizzle(row & 15)) << 4);
  }
  uint32_t read_at[NT], swizzle[NT];  // of the lane's token
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rows = min(FOURS * 4 - nt * 16, 16), row = nt * 16 + (r & (rows - 1));  // 4, 8 or 16 rows: others repeat
    read_at[nt] = row * 256;
    swizzle[nt] = token_swizzle(row & 15);
  }
  uint16_t* act[NT];  // where the lane's tokens' activations go (a row past the last: not used)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int token = min(nt * 16 + r, count - 1), first = token / TILE_TOKENS * TILE_TOKENS;
    const int to = act_tile(p, expert, number + first / TILE_TOKENS, slots[first]);
    act[nt] = p.act + (size_t)to * 2 * TOKENS * p.inner + token % TILE_TOKENS * 16;
  }
  int t_next = 0;
  auto load_tokens = [&](int i) {
    const int block = step_of(i / BLOCKS) * BLOCKS + i % BLOCKS;
#pragma unroll
    for (int q = 0; q < FOURS; ++q) dma16(x, x_at[q], (uint32_t)block * 256, token_base + t_next * TOKEN_BYTES + q * 1024);
    t_next = t_next == T_SLOTS - 1 ? 0 : t_next + 1;
  };

  auto first_tokens = [&]() {
    t_next = 0;
#pragma unroll
    for (int i = 0; i < T_AHEAD; ++i)
      if (i < blocks) load_tokens(i);
  };

  int w_slot = 0;
  first_tokens();
  for (; tile < tile_end; ++tile) {
    f32x4 acc[TILES][NT];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[i][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    int t_slot = 0;
    // Block by block: its tokens' loads go T_AHEAD blocks ahead, those of the weights a step.
    auto multiply = [&](int i, auto BLOCK) {
      constexpr int block = decltype(BLOCK)::value;
      // In this order what may still be on its way is the next step's weights and the tokens
      // of the blocks after this, whichever came first.
      before_loads();
      if constexpr (BLOCKS == 1) load_weights();
      if (i + T_AHEAD < blocks) load_tokens(i + T_AHEAD);
      if constexpr (BLOCKS == 2 && block == 0) load_weights();
      const int tokens_after = min(T_AHEAD, blocks - 1 - i);
      if (tokens_after == 0) wait_loads<W>();
      else if (tokens_after == 1) wait_loads<W + T>();
      else wait_loads<W + T_AHEAD * T>();
      const uint8_t* const st = ring + w_slot * STEP;
      const uint8_t* const tok = ring + UP_W_SLOTS * STEP + t_slot * TOKEN_BYTES;
      u32x4 t[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t piece = FP4 ? 4 * g + j : 8 * (j >> 1) + 2 * g + (j & 1);
          t[nt][j] = *reinterpret_cast<const u32x4*>(tok + read_at[nt] + ((piece ^ swizzle[nt]) << 4));
        }
#pragma unroll
      for (int k = 0; k < TILES; ++k) weights.template multiply<NT>(acc[k], st, k, block, t, lane);
      t_slot = t_slot == T_SLOTS - 1 ? 0 : t_slot + 1;
    };
    for (int i = 0; i < steps; ++i) {
      multiply(i * BLOCKS, std::integral_constant<int, 0>{});
      if constexpr (BLOCKS == 2)
        if (i * 2 + 1 < blocks) multiply(i * 2 + 1, std::integral_constant<int, 1>{});
      w_slot = w_slot == UP_W_SLOTS - 1 ? 0 : w_slot + 1;
    }

    before_loads();
    if (tile + 1 < tile_end) first_tokens();
    auto sums_of = [&](int w) { return reinterpret_cast<f32x4*>(lds + w * UP_RING<FP4, RT> + SUMS_AT); };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < TILES; ++i) sums_of(wave)[(nt * TILES + i) * 64 + lane] = acc[i][nt];
    meet();
    for (int item = wave; item < RT * NT; item += UP_WAVES) {
      const int nt = item / RT, i = item % RT, at = nt * TILES + i;
      f32x4 gate = sums_of(0)[at * 64 + lane], up = sums_of(0)[(at + RT) * 64 + lane];
#pragma unroll
      for (int w = 1; w < UP_WAVES; ++w) {
        gate += sums_of(w)[at * 64 + lane];
        up += sums_of(w)[(at + RT) * 64 + lane];
      }
      f32x4 a;
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = gate[k] * sigmoid(gate[k]) * up[k];
      if (nt * 16 + r < count) {
        uint16_t* to = act[0];  // (a choice by an index would put them in memory)
        if constexpr (NT > 1) to = nt ? act[1] : to;
        const int k = tile * 16 * RT + 16 * i + 4 * g;
        *reinterpret_cast<u32x2*>(to + act_at<FP4, TOKENS>(k, 0)) = (u32x2){upper2(a[0], a[1]), upper2(a[2], a[3])};
        *reinterpret_cast<u32x2*>(to + act_at<FP4, TOKENS>(k, 1)) = (u32x2){lower2(a[0], a[1]), lower2(a[2], a[3])};
      }
    }
    meet();  // the sums have been read: tokens may come
  }
  wait_loads<0>();  // (the last step's weights once more)
  meet();
}

// The tiles of all experts that have tokens, in order, are dealt to the workgroups in
// runs of the same length. The first workgroup writes the plan as well.
template <bool FP4, int RT, int TOKENS>
__global__ __launch_bounds__(UP_THREADS, 1) void experts_up_kernel(ExpertsArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[UP_WAVES * UP_RING<FP4, RT>];
  __shared__ UpLists l;
  static_assert(UP_WAVES * UP_RING<FP4, RT> >= 2 * MAX_GROUPS * 4, "the tables of groups in the rings' place");
  const int n = p.tokens * p.top_k, tid = threadIdx.x, lane = tid & 63;
  int* const first = reinterpret_cast<int*>(lds);  // of each group's slots
  for (int i = tid; i < n; i += UP_THREADS) {
    const int e = p.ids[i];
    l.ids[i] = (short)(e >= 0 && e < p.num_groups ? e : -1);
  }
  for (int e = tid; e < p.num_groups; e += UP_THREADS) first[e] = n;
  meet();
  for (int i = tid; i < n; i += UP_THREADS)
    if (l.ids[i] >= 0) atomicMin(&first[l.ids[i]], i);
  meet();
  const int experts = gather(l, n, [&](int i) { return l.ids[i] >= 0 && first[l.ids[i]] == i; },
                             [&](int i, int at) { l.active[at] = (uint16_t)l.ids[i]; });
  if (blockIdx.x == 0) {
    if (tid < 64) write_plan(p, l, experts, first, first + MAX_GROUPS);
    meet();
  }

  const int tiles = p.inner / (16 * RT), all = experts * tiles;  // at most 2^22
  const int grid = gridDim.x, share = all / grid, more = all % grid, b = blockIdx.x;
  int at = b * share + min(b, more);
  const int end = at + share + (b < more);
  UpWeights<FP4, RT> weights(p.b1, p.sfb1, 2 * p.inner, p.hidden, lane);
  while (at < end) {
    const int expert = __builtin_amdgcn_readfirstlane((int)l.active[at / tiles]);
    const int tile = at % tiles, tile_end = min(tile + end - at, tiles);
    at += tile_end - tile;
    const int count = gather(l, n, [&](int i) { return l.ids[i] == expert && first_of_token(l.ids, i, p.top_k); },
                             [&](int i, int place) { l.list[place] = (uint16_t)i; });
    // The tokens 32 at a time.
    for (int t0 = 0; t0 < count;) {
      const int left = count - t0, here = min(left, 4 * UP_MOST_FOURS);
      const uint16_t* const slots = l.list + t0;
      const int number = t0 / TILE_TOKENS;
      if constexpr (TOKENS == 4) {
        up_tiles<FP4, RT, 1, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
      } else {
        if (here <= 4) up_tiles<FP4, RT, 1, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
        else if (here <= 8) up_tiles<FP4, RT, 2, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
        else if (here <= 16) up_tiles<FP4, RT, 4, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
        else if (here <= 24) up_tiles<FP4, RT, 6, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
        else up_tiles<FP4, RT, 8, TOKENS>(p, weights, tile, tile_end, expert, number, slots, here, lds);
      }
      t0 += here;
    }
  }
}

// ---------------------------------------------------------------------------
// Down
// ---------------------------------------------------------------------------

constexpr int DOWN_WAVES = 4, DOWN_THREADS = DOWN_WAVES * 64;

// Steps on their way and in use: as many as leave the sums and the operands' registers room.
template <bool FP4, int NT>
constexpr int DOWN_DEPTH = (FP4 ? 4 : 5) - (NT == 4 ? 2 : NT == 2 ? 1 : 0);
template <bool FP4, int RT>
using DownWeights = Weights<FP4, RT, 1>;

// Of the other lane of a pair (DPP quad_perm 1, 0, 3, 2).
__device__ __forceinline__ float neighbour(float v) {
  return __builtin_bit_cast(float, quad<0xB1>(__builtin_bit_cast(uint32_t, v)));
}

struct DownItem {
  int expert_count, begin, tile;  // pairs of the plan (expert << 8 | how many), and their first activations
};

// A workgroup takes 16 RT columns of y for all tokens (of which a call has at most MOST).
// Its waves share the experts, NT tiles of 8 tokens of one at a time (NT is as many as the
// call's tokens fill, up to 4), and, where these do not come out even, their K in parts; each
// wave keeps sums of its own in LDS, which are added in order at the end. A wave's items
// follow one another in one pipeline of steps.
template <bool FP4, int TOKENS, int MOST, int NT, int RT>
__global__ __launch_bounds__(DOWN_THREADS, 1) void experts_down_kernel(ExpertsArgs p) {
  constexpr int STRIDE = 16 * RT + (MOST > 64 ? 0 : 4);  // floats; 4 past a power of two where there is room
  constexpr int DEPTH = DOWN_DEPTH<FP4, NT>, W = DownWeights<FP4, RT>::LOADS, STEP = DownWeights<FP4, RT>::BYTES;
  // Loads of activations in a step: at least one tile's.
  constexpr int BLOCKS = DownWeights<FP4, RT>::BLOCKS, ACT_LOADS = 4 * BLOCKS;
  __shared__ __attribute__((aligned(1024))) uint8_t rings[DOWN_WAVES * DEPTH * STEP];
  __shared__ __attribute__((aligned(16))) float sums[DOWN_WAVES * MOST * STRIDE];
  // Of the pairs; read from memory in the loop, they would be waited for with all the
  // weights that are on their way.
  __shared__ DownItem items[MAX_FEW_PAIRS];
  __shared__ uint16_t slots[MAX_FEW_PAIRS];    // the pair's slot,
  __shared__ uint16_t sums_at[MAX_FEW_PAIRS];  // where its token's sums are, in 16 bytes
  __shared__ float pair_weights[MAX_FEW_PAIRS];
  __shared__ int items_of[DOWN_WAVES];
  __shared__ bool last;
  ExpertPlan* const plan = reinterpret_cast<ExpertPlan*>(p.plan);
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), c0 = blockIdx.x * 16 * RT;
  float* const mine = sums + wave * MOST * STRIDE;
  for (int i = lane; i < p.tokens * STRIDE; i += 64) mine[i] = 0.0f;

  // What the plan may hold is read before it is known how much of that it does hold: one
  // way to memory, not three.
  const int n = p.tokens * p.top_k, most = min(n, p.num_groups), experts = plan->experts;
  for (int i = tid; i < n; i += DOWN_THREADS) {
    const int slot = plan->slot[i];
    slots[i] = (uint16_t)slot;
    sums_at[i] = (uint16_t)(slot / p.top_k * (STRIDE / 4));
    pair_weights[i] = plan->weight[i];
  }
  // The items: an expert's pairs 8 NT at a time, in order.
  constexpr int ITEM = TILE_TOKENS * NT;
  int total = 0;
  for (int r0 = 0; r0 < most; r0 += DOWN_THREADS) {
    const int at = r0 + tid;
    const ExpertEntry entry = plan->entry[min(at, most - 1)];
    const int has = at < experts ? (entry.count + ITEM - 1) / ITEM : 0;
    int upto = has;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) items_of[wave] = upto;
    __syncthreads();
    int before = total + upto - has;
    for (int w = 0; w < DOWN_WAVES; ++w) {
      if (w < wave) before += items_of[w];
      total += items_of[w];
    }
    for (int i = 0; i < has; ++i) {
      const int begin = entry.begin + ITEM * i, count = min(entry.count - ITEM * i, ITEM);
      const int tile = act_tile(p, entry.expert, NT * i, i == 0 ? entry.first : plan->slot[begin]);
      items[before + i] = DownItem{entry.expert << 8 | count, begin, tile};
    }
    __syncthreads();
  }
  total = __builtin_amdgcn_readfirstlane(total);

  // Parts of K: so many that the waves have the same number of items, or that they have
  // eight each. The workgroups of the same columns share them like waves.
  const int waves = DOWN_WAVES * p.splits, me = blockIdx.y * DOWN_WAVES + wave;
  const int item_steps = (p.inner / QBLOCK + BLOCKS - 1) / BLOCKS;
  int parts = 1;
  while (parts < 8 && parts * 2 <= item_steps && total * parts % waves && total * parts < 8 * waves) parts *= 2;
  const int all = total * parts, turns = me < all ? (all - me + waves - 1) / waves : 0;

  // Where the loads and the products are: the turn, its item and its steps.
  struct Cursor {
    int turn, step, end, begin, count, tile;
  };
  auto start = [&](Cursor& c) {
    const int item = me + c.turn * waves, part = item % parts;
    const DownItem at = items[item / parts];
    c.begin = __builtin_amdgcn_readfirstlane(at.begin);
    c.tile = __builtin_amdgcn_readfirstlane(at.tile);
    const int expert_count = __builtin_amdgcn_readfirstlane(at.expert_count);
    c.count = expert_count & 0xFF;
    c.step = item_steps * part / parts;
    c.end = item_steps * (part + 1) / parts;
    return expert_count >> 8;
  };
  int steps = 0;
  for (int turn = 0; turn < turns; ++turn) {
    const int part = (me + turn * waves) % parts;
    steps += item_steps * (part + 1) / parts - item_steps * part / parts;
  }

  if (steps > 0) {
    const uint8_t* const ring = rings + wave * DEPTH * STEP;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_void*)ring;
    const int row0[1] = {c0};
    Cursor ahead{}, now{};
    start(now);
    const int first = start(ahead);
    DownWeights<FP4, RT> weights(p.b2, p.sfb2, p.hidden, p.inner, lane);
    weights.place(first, row0, lane);
    // The item's activations: lanes 2 t and 2 t + 1 load the two parts of a token's. Rows past
    // its pairs are not loaded (they lie past the end, as does a second block past the last).
    __amdgpu_buffer_rsrc_t act[NT];
    uint32_t act_at[NT];
    auto place_act = [&]() {
      const uint32_t tile_values = (uint32_t)(2 * TOKENS) * p.inner;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int first = TILE_TOKENS * nt, token = first + r / 2;
        int tile = ahead.tile;
        if (nt > 0 && first < ahead.count) tile = tiles_by_slot(p) ? slots[ahead.begin + first] : tile + nt;
        act[nt] = buffer_rsrc(p.act + (size_t)tile * tile_values, tile_values * 2);
        act_at[nt] = token < ahead.count ? (uint32_t)(g * 2 * TOKENS + r) * 16 : 0x80000000u;
      }
    };
    place_act();
    f32x4 acc[RT][NT] = {};
    int loaded = 0, w_next = 0, w_slot = 0;
    u32x4 t[DEPTH][BLOCKS][NT][4];
    auto load = [&](u32x4 (&to)[BLOCKS][NT][4]) __attribute__((always_inline)) {
      // Tiles that the item does not have are not asked for: a load takes its turn at the L1
      // whether it has rows or not (57 tokens, 82 experts of 1536 x 1536: 184 us for 148).
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt == 0 || TILE_TOKENS * nt < ahead.count) {
#pragma unroll
          for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              to[b][nt][j] = __builtin_amdgcn_raw_buffer_load_b128(
                  act[nt], act_at[nt] + (b * QBLOCK + j * 32) * TOKENS * 4, ahead.step * BLOCKS * QBLOCK * TOKENS * 4, 0);
        }
      weights.load(ahead.step, base + w_next * STEP);
      w_next = w_next == DEPTH - 1 ? 0 : w_next + 1;
      if (++loaded < steps && ++ahead.step == ahead.end) {  // (past the last step it is loaded again)
        ++ahead.turn;
        const int e = start(ahead);
        weights.place(e, row0, lane);
        place_act();
      }
    };
    auto use = [&](const u32x4 (&from)[BLOCKS][NT][4]) __attribute__((always_inline)) {
      const uint8_t* const st = ring + w_slot * STEP;
      w_slot = w_slot == DEPTH - 1 ? 0 : w_slot + 1;
      // As many tiles as the item has.
      auto multiply = [&](auto TILES) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
          for (int k = 0; k < RT; ++k)
            weights.template multiply<decltype(TILES)::value>(acc[k], st, k, b, from[b], lane);
      };
      if (NT > 3 && now.count > 3 * TILE_TOKENS) multiply(std::integral_constant<int, NT>{});
      else if (NT > 2 && now.count > 2 * TILE_TOKENS) multiply(std::integral_constant<int, std::min(NT, 3)>{});
      else if (NT > 1 && now.count > TILE_TOKENS) multiply(std::integral_constant<int, std::min(NT, 2)>{});
      else multiply(std::integral_constant<int, 1>{});
      if (++now.step < now.end) return;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // The sums of the lower parts to those of the upper ones.
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[k][nt][v] += neighbour(acc[k][nt][v]);
        const int pair = TILE_TOKENS * nt + r / 2;
        if (r % 2 == 0 && pair < now.count) {  // the item's tokens differ from one another
          const float w = pair_weights[now.begin + pair];
          float* const at = mine + 4 * (sums_at[now.begin + pair] + g);
#pragma unroll
          for (int k = 0; k < RT; ++k) {
            f32x4 sum = *reinterpret_cast<f32x4*>(at + 16 * k);
#pragma unroll
            for (int v = 0; v < 4; ++v) sum[v] = __builtin_fmaf(w, acc[k][nt][v], sum[v]);
            *reinterpret_cast<f32x4*>(at + 16 * k) = sum;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < RT; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[k][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};
      if (++now.turn < turns) start(now);
    };
    // Rounds that are left at their end only, so that on every path to a use the compiler
    // knows how many loads follow the ones that it waits for: those of steps with one tile
    // (the waits for the weights go by these as well).
    static_for<0, DEPTH - 1>([&](auto I) { load(t[decltype(I)::value]); });
    const int rounds = steps / DEPTH * DEPTH;
    for (int i0 = 0; i0 < rounds; i0 += DEPTH) {
      static_for<0, DEPTH>([&](auto I) {
        constexpr int j = decltype(I)::value;
        before_loads();
        load(t[(j + DEPTH - 1) % DEPTH]);
        wait_loads<(DEPTH - 1) * (ACT_LOADS + W)>();
        use(t[j]);
      });
    }
    wait_loads<0>();
    static_for<0, DEPTH - 1>([&](auto I) {
      if (rounds + decltype(I)::value < steps) use(t[decltype(I)::value]);
    });
  }
  __syncthreads();
  for (int i = tid; i < p.tokens * 8 * RT; i += DOWN_THREADS) {
    const int t = i / (8 * RT), c = i % (8 * RT) * 2;
    f32x2 s = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < DOWN_WAVES; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) s[k] += sums[(w * MOST + t) * STRIDE + c + k];
    if (p.splits == 1)
      *reinterpret_cast<uint32_t*>(p.y + (size_t)t * p.hidden + c0 + c) = pack2(s);
    else
      __hip_atomic_store(reinterpret_cast<uint64_t*>(p.partial + ((size_t)blockIdx.y * p.tokens + t) * p.hidden + c0 + c),
                         __builtin_bit_cast(uint64_t, s), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (p.splits == 1) return;
  // The last of the columns' workgroups to be done adds their sums, in order. They go
  // past the L2s by accesses of agent scope, and are there once waited for: a fence would
  // write back and drop a whole L2 for each workgroup (20 us of 50).
  wait_vmcnt_0();
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(&plan->done[blockIdx.x], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
  __syncthreads();
  if (!last) return;
  for (int i = tid; i < p.tokens * 8 * RT; i += DOWN_THREADS) {
    const int t = i / (8 * RT), c = i % (8 * RT) * 2;
    f32x2 s = {0.f, 0.f};
    for (int w = 0; w < p.splits; ++w) {
      const f32x2 v = __builtin_bit_cast(
          f32x2, __hip_atomic_load(reinterpret_cast<uint64_t*>(p.partial + ((size_t)w * p.tokens + t) * p.hidden + c0 + c),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
      for (int k = 0; k < 2; ++k) s[k] += v[k];
    }
    *reinterpret_cast<uint32_t*>(p.y + (size_t)t * p.hidden + c0 + c) = pack2(s);
  }
}

template <bool FP4, int RT, int TOKENS>
hipError_t launch_up(const ExpertsArgs& a, hipStream_t stream) {
  const int workgroups = std::min(std::min(a.tokens * a.top_k, a.num_groups) * (a.inner / (16 * RT)), a.cus);
  hipLaunchKernelGGL((experts_up_kernel<FP4, RT, TOKENS>), dim3(workgroups), dim3(UP_THREADS), 0, stream, a);
  return hipGetLastError();
}

template <bool FP4, int TOKENS, int MOST, int NT>
hipError_t launch_down(const ExpertsArgs& a, hipStream_t stream) {
  // 16 columns a workgroup, and the activations read twice as often, where 32 would leave
  // half the compute units without one. 128 tokens, 64 experts of 4096 x 1536 in FP8: 121
  // us, with 32 columns 186; 16 tokens: 72 and 100. With hidden 7168 (448 workgroups for
  // 224) 61 tokens and 32 experts took 198 us for 129.
  const int rt = a.hidden / 32 <= a.cus / 2 ? 1 : 2;
  const auto down = rt == 1 ? experts_down_kernel<FP4, TOKENS, MOST, NT, 1> : experts_down_kernel<FP4, TOKENS, MOST, NT, 2>;
  hipLaunchKernelGGL(down, dim3(a.hidden / (16 * rt), a.splits), dim3(DOWN_THREADS), 0, stream, a);
  return hipGetLastError();
}

// How many workgroups of the second launch share the experts of their columns: as many as
// there is room for, while each wave keeps eight steps. Whole layers, in us, with and
// without: 57 tokens, 82 experts of 1536 x 1536 in FP8 135, 175; 8 tokens, 43 experts of
// 768 x 1664 in FP4 38, 56; 5 tokens, 26 experts of 512 x 896 in FP8 25, 33. (Not by the
// compute units that are set: the order of the sums differs.)
int down_splits(const ExpertsArgs& a) {
  const int experts = std::min(a.tokens * a.top_k, a.num_groups), steps = a.inner / (a.fp4 ? 2 * QBLOCK : QBLOCK);
  return std::max(std::min(DOWN_COLUMNS / a.hidden, experts * steps / (8 * DOWN_WAVES)), 1);
}

// TOKENS: 4 for up to 4 tokens, else 8.
template <bool FP4, int TOKENS>
hipError_t launch_both(const ExpertsArgs& a, hipStream_t stream) {
  // Half as many rows a workgroup where there would not be one for every compute unit.
  const bool few = std::min(a.tokens * a.top_k, a.num_groups) * (a.inner / 32) < a.cus;
  if (hipError_t e = few ? launch_up<FP4, 1, TOKENS>(a, stream) : launch_up<FP4, 2, TOKENS>(a, stream)) return e;
  if constexpr (TOKENS == 4) return launch_down<FP4, TOKENS, 4, 1>(a, stream);
  else if (a.tokens <= 8) return launch_down<FP4, TOKENS, 64, 1>(a, stream);
  else if (a.tokens <= 16) return launch_down<FP4, TOKENS, 64, 2>(a, stream);
  else if (a.tokens <= 64) return launch_down<FP4, TOKENS, 64, 4>(a, stream);
  else return launch_down<FP4, TOKENS, MAX_FEW_TOKENS, 4>(a, stream);
}

}  // namespace

long long experts_act_bytes(int tokens, int top_k, int num_groups, int inner) {
  const int n = tokens * top_k, tiles = n <= num_groups ? n : num_groups * ((tokens + TILE_TOKENS - 1) / TILE_TOKENS);
  return (long long)tiles * (tokens <= 4 ? 4 : TILE_TOKENS) * inner * 4;
}

hipError_t launch_experts(ExpertsArgs a, hipStream_t stream) {
  a.splits = down_splits(a);
  if (a.tokens <= 4) return a.fp4 ? launch_both<true, 4>(a, stream) : launch_both<false, 4>(a, stream);
  return a.fp4 ? launch_both<true, 8>(a, stream) : launch_both<false, 8>(a, stream);
}

}  // namespace moe
}  // namespace dg
