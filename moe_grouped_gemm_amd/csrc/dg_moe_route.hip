// Tokens sorted by expert into the GEMMs' row layouts, moved there (BF16, or
// quantised to the FP8 operand) and back with weights, and the gradients.

#include <algorithm>

#include "dg_moe_device.h"

namespace dg {
namespace moe {
namespace {

// Lanes of the wave that hold the same key as this one (`valid` ones only):
// one ballot per key bit.
__device__ __forceinline__ uint64_t same_key(int key, bool valid, int bits) {
  uint64_t m = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const uint64_t ones = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? ones : ~ones;
  }
  return m;
}

// Sorting by counting, in two passes over chunks of the slots: the first
// counts each chunk's ids per group, the second finds from all the counts
// where each group starts and how many of its rows come before the chunk, and
// ranks the chunk's slots. Within a wave equal ids are ranked by ballots; the
// waves take turns to advance the groups' next free rows, which keeps the
// order. Bound by latency: 2 N reads and N writes of 4 bytes are nothing, so
// chunks are as small as keeps the table of counts small (MAX_CHUNKS rows,
// read by every workgroup of the second pass). 65536 slots over 32 groups take
// 5 and 7 us, in one workgroup they took 174.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int MAX_CHUNKS = 256;

__host__ __device__ inline int chunk_slots(int slots) {
  const int per = (slots + MAX_CHUNKS - 1) / MAX_CHUNKS;
  return per <= SORT_THREADS ? SORT_THREADS : (per + SORT_THREADS - 1) / SORT_THREADS * SORT_THREADS;
}

// First row of each group from the groups' sizes, by the whole workgroup;
// writes group_rows where asked. A barrier ends it.
template <int THREADS>
__device__ void group_starts(const RouteArgs& p, const int* total, int* first, bool write_rows) {
  __shared__ int scan[THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int rows_before = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += THREADS) {
    const int g = g0 + tid;
    const int count = g < p.num_groups ? total[g] : 0;
    const int size = p.layout == DG_MOE_CONTIGUOUS ? (count + SEGMENT - 1) / SEGMENT * SEGMENT : count;
    int incl = size;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 63) scan[wave] = incl;
    __syncthreads();
    int waves_before = 0, sum = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < wave) waves_before += scan[w];
      sum += scan[w];
    }
    if (g < p.num_groups) {
      const int start = p.layout == DG_MOE_MASKED ? g * p.rows : rows_before + waves_before + incl - size;
      const int room = p.layout == DG_MOE_MASKED ? p.rows : max(p.rows - start, 0);
      first[g] = start;
      if (write_rows) p.group_rows[g] = min(count, room);
    }
    rows_before += sum;
    __syncthreads();
  }
}

// The contiguous layout's group of each row begin, begin + step, ...
__device__ void fill_layout(const RouteArgs& p, const int* total, const int* first, int begin, int step) {
  for (int r = begin; r < p.rows; r += step) {
    int lo = 0, hi = p.num_groups - 1;  // last group that starts at or before r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= r) lo = mid; else hi = mid - 1;
    }
    p.grouped_layout[r] = r >= first[lo] && r < first[lo] + total[lo] ? lo : -1;
  }
}

__global__ __launch_bounds__(SORT_THREADS) void count_kernel(RouteArgs p, int chunk) {
  __shared__ int count[MAX_GROUPS];
  const int tid = threadIdx.x, G = p.num_groups, N = p.tokens * p.top_k;
  for (int g = tid; g < G; g += SORT_THREADS) count[g] = 0;
  __syncthreads();
  const int begin = blockIdx.x * chunk, end = min(begin + chunk, N);
  for (int i = begin + tid; i < end; i += SORT_THREADS) {
    const int e = p.ids[i];
    if (e >= 0 && e < G) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  int* out = static_cast<int*>(p.workspace) + (size_t)blockIdx.x * G;
  for (int g = tid; g < G; g += SORT_THREADS) out[g] = count[g];
}

__global__ __launch_bounds__(SORT_THREADS) void rank_kernel(RouteArgs p, int chunk, int chunks) {
  __shared__ int next[MAX_GROUPS];   // rows of the group before this chunk, then its next free row
  __shared__ int total[MAX_GROUPS];  // rows of the group
  __shared__ int first[MAX_GROUPS];  // first row of the group
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G = p.num_groups, N = p.tokens * p.top_k;
  const int* counts = static_cast<const int*>(p.workspace);

  for (int g = tid; g < G; g += SORT_THREADS) next[g] = total[g] = 0;
  __syncthreads();
  const int begin = blockIdx.x * chunk, end = min(begin + chunk, N);
  // The table of counts, summed over chunks: as many chunks at once as there
  // are threads for.
  int width = 1;
  while (width < G && width < SORT_THREADS) width <<= 1;
  const int slices = SORT_THREADS / width, slice = tid / width;
  for (int g = tid & (width - 1); g < G; g += width) {
    int before = 0, all = 0;
#pragma unroll 4
    for (int c = slice; c < chunks; c += slices) {
      const int v = counts[(size_t)c * G + g];
      all += v;
      before += c < (int)blockIdx.x ? v : 0;
    }
    if (all) {
      atomicAdd(&total[g], all);
      atomicAdd(&next[g], before);
    }
  }
  __syncthreads();

  group_starts<SORT_THREADS>(p, total, first, blockIdx.x == 0);
  for (int g = tid; g < G; g += SORT_THREADS) next[g] += first[g];  // (each read below by a later barrier)

  const int bits = 32 - __builtin_clz(G);
  for (int i0 = begin; i0 < end; i0 += SORT_THREADS) {
    const int i = i0 + tid;
    const int e = i < end ? p.ids[i] : -1;
    const bool valid = e >= 0 && e < G;
    const uint64_t peers = same_key(e, valid, bits);
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    int base = 0;
    for (int w = 0; w < SORT_WAVES; ++w) {
      __syncthreads();
      if (w == wave && valid) {
        base = next[e];
        if (rank == 0) next[e] = base + __popcll(peers);
      }
    }
    if (i < end) {
      const int row = base + rank;
      const bool fits = valid && row < (p.layout == DG_MOE_MASKED ? (e + 1) * p.rows : p.rows);
      p.row_of[i] = fits ? row : -1;
    }
  }

  if (p.layout == DG_MOE_CONTIGUOUS)
    fill_layout(p, total, first, blockIdx.x * SORT_THREADS + tid, chunks * SORT_THREADS);
}

constexpr int DISPATCH_THREADS = 512;  // 256: 65536 rows of 7168 in FP8 take 4% more time, BF16 rows the same

// How a token's values arrive in its rows: copied, or quantised with float32
// or power-of-two scales (or not at all, where only the sort is wanted).
enum { MOVE_BF16 = 0, MOVE_FP8 = 1, MOVE_FP8_E8 = 2, MOVE_NONE = 3 };

struct MoveArgs {
  const uint16_t* x;
  uint8_t* out;  // rows of BF16 or E4M3
  float* sfa;    // quantised only
};

// Block b (128 values) of token t to the rows of up to 16 slots: 16 lanes, 8
// values each; lane l16 of the 16 has the row of slot l16 or -1.
template <int MODE>
__device__ __forceinline__ void put_block(const RouteArgs& p, const MoveArgs& m, u32x4 raw, int b, int l16, int row,
                                          int slots) {
  constexpr int BYTES = MODE == MOVE_BF16 ? 2 : 1;
  const size_t offset = ((size_t)b * QBLOCK + l16 * 8) * BYTES, stride = (size_t)p.hidden * BYTES;
  u32x2 codes;
  if constexpr (MODE != MOVE_BF16) {
    float scale;
    codes = quantize_row<MODE == MOVE_FP8_E8>(unpack8(raw), scale);
    // Lane l16 leaves the scale of slot l16.
    if (row >= 0) {
      const int blocks = p.hidden / QBLOCK, ld = align4(p.rows);
      const int g = p.layout == DG_MOE_MASKED ? row / p.rows : 0;
      m.sfa[((size_t)g * blocks + b) * ld + (row - g * p.rows)] = scale;
    }
  }
  static_for<0, 16>([&](auto J) {
    constexpr int j = decltype(J)::value;
    if (j >= slots) return;
    const int r = bcast16<j>(row);
    if (r < 0) return;
    if constexpr (MODE == MOVE_BF16) store_stream(m.out + (size_t)r * stride + offset, raw);
    else store_stream(m.out + (size_t)r * stride + offset, codes);
  });
}

// Tokens to rows: 16 lanes a block of 128 values, read (and quantised) once
// and written to the rows of the token's slots. Bound by memory, mostly
// writes. Each XCD takes a contiguous range of tokens: the scales of a
// group's consecutive rows, which lie side by side in sfa, then meet in one
// L2, and as the codes are stored past it, stay there until their lines are
// full: 65536 rows of 7168 in FP8 write 462 MiB, which is what they are, in 120
// us (5.0 TB/s with the tokens read); without the scales, which are stored 4
// bytes at a time, it would be 10 us less. 26500 BF16 rows: 90 us (5.4 TB/s).
template <int MODE>
__global__ __launch_bounds__(DISPATCH_THREADS) void dispatch_kernel(RouteArgs p, MoveArgs m) {
  const int blocks = p.hidden / QBLOCK, l16 = threadIdx.x & 15;
  const int tokens_per = (p.tokens + 7) / 8;
  const int t0 = (blockIdx.x & 7) * tokens_per, here = min(tokens_per, p.tokens - t0);
  if (here <= 0) return;
  // Block i of the XCD's tokens (fewer than 2^30: the tokens take less than
  // 2^40 bytes); a grid at its cap goes round again.
  const uint32_t end = (uint32_t)here * blocks;
  for (uint32_t i = (blockIdx.x >> 3) * (DISPATCH_THREADS / 16) + (threadIdx.x >> 4); i < end;
       i += (gridDim.x >> 3) * (DISPATCH_THREADS / 16)) {
    const int t = t0 + (int)(i / (uint32_t)blocks), b = (int)(i % (uint32_t)blocks);
    const uint16_t* src = m.x + (size_t)t * p.hidden + b * QBLOCK + l16 * 8;
    const u32x4 raw = MODE == MOVE_BF16 ? load16(src) : load_stream16(src);
    for (int j0 = 0; j0 < p.top_k; j0 += 16) {
      const int slots = min(p.top_k - j0, 16);
      const int row = l16 < slots ? p.row_of[(size_t)t * p.top_k + j0 + l16] : -1;
      put_block<MODE>(p, m, raw, b, l16, row, slots);
    }
  }
}

// Few slots: one launch sorts and moves. A workgroup takes a few tokens, counts
// all the ids itself -- those of the slots before its own, and all of them --
// finds the groups' starts from the counts, ranks its own slots as rank_kernel
// does and moves its tokens; in the contiguous layout every workgroup writes a
// share of the rows' groups, and there may be workgroups without tokens for that.
// Bound by latency: a launch costs more than the counting, which is the same in
// every workgroup, LDS atomics on whole numbers (their order does not matter)
// that grow with the slots. An XCD takes successive tokens, for their rows' scales
// as in dispatch_kernel (without that 8192 slots of 7168 values took a seventh more). Ranking by
// comparing each slot with all ids took as long at 40 slots and 14 us at 4096.
// Where it is used: one_launch.
constexpr int FEW_SLOTS = 16384;  // at most
constexpr int FEW_THREADS = 512;
constexpr int FEW_WORKGROUPS = 512;  // 256: slower with long rows, 1024: with many slots
constexpr int FILL_ROWS = 2048;      // rows of grouped_layout that are worth a workgroup
// A workgroup's slots are at most its share of them and one token's more.
static_assert(FEW_SLOTS / FEW_WORKGROUPS + MAX_TOP_K <= 64, "a wave ranks a workgroup's slots");

// Counters in LDS for few groups come in several copies, a lane's one by its number, so
// that lanes with the same id seldom meet in one atomic: 8192 ids over 2 groups (rows
// of 256) take 7.7 us, with one copy 17.2, over 4 groups 7.5 and 10.9; 4096 ids over
// 32 groups 6.2 and 5.7. Many groups spread by themselves if the ids do, and few ids are
// not worth clearing and adding up more counters.
__device__ __forceinline__ int counter_copies(int ids, int groups) {
  int copies = 1;
  while (copies * groups < 64 && copies * 1024 < ids) copies <<= 1;
  return copies;  // copies * groups < 128, or 1
}
// The copies' sum for group g, left in its first counter.
__device__ __forceinline__ void sum_copies(int* counters, int copies, int groups, int g) {
  int s = 0;
  for (int c = 0; c < copies; ++c) s += counters[c * groups + g];
  counters[g] = s;
}

template <int MODE>
__global__ __launch_bounds__(FEW_THREADS) void few_kernel(RouteArgs p, MoveArgs m, int tokens_each) {
  __shared__ int next[MAX_GROUPS];   // rows of the group before these tokens, then its next free row
  __shared__ int total[MAX_GROUPS];  // rows of the group
  __shared__ int first[MAX_GROUPS];  // first row of the group
  __shared__ int rows[64];           // of this workgroup's slots
  const int tid = threadIdx.x, l16 = tid & 15;
  const int G = p.num_groups, N = p.tokens * p.top_k, k = p.top_k;
  const int chunk = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int t0 = chunk * tokens_each, tokens = max(min(tokens_each, p.tokens - t0), 0);
  const int begin = t0 * k, slots = tokens * k;

  // On their way while the ids are counted: the first piece of the tokens, the
  // workgroup's own ids.
  const int blocks = p.hidden / QBLOCK, first_item = tid >> 4;
  u32x4 raw = {};
  if (MODE != MOVE_NONE && first_item < tokens * blocks)
    raw = load16(m.x + (size_t)t0 * p.hidden + first_item * QBLOCK + l16 * 8);
  const int e = tid < slots ? p.ids[begin + tid] : -1;

  const int copies = counter_copies(N, G), mine = (tid & (copies - 1)) * G;
  for (int g = tid; g < copies * G; g += FEW_THREADS) next[g] = total[g] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < N; i += FEW_THREADS) {
    const int id = p.ids[i];
    if (id < 0 || id >= G) continue;
    atomicAdd(&total[mine + id], 1);
    if (i < begin) atomicAdd(&next[mine + id], 1);
  }
  __syncthreads();
  if (copies > 1) {
    for (int g = tid; g < G; g += FEW_THREADS) {
      sum_copies(total, copies, G, g);
      sum_copies(next, copies, G, g);
    }
    __syncthreads();
  }
  if (p.layout == DG_MOE_MASKED) {
    for (int g = tid; g < G; g += FEW_THREADS) {
      next[g] += g * p.rows;
      if (blockIdx.x == 0) p.group_rows[g] = min(total[g], p.rows);
    }
  } else {
    group_starts<FEW_THREADS>(p, total, first, blockIdx.x == 0);
    for (int g = tid; g < G; g += FEW_THREADS) next[g] += first[g];
  }
  __syncthreads();

  if (tid < 64) {
    const bool valid = e >= 0 && e < G;
    const uint64_t peers = same_key(e, valid, 32 - __builtin_clz(G));
    int row = -1;
    if (valid) {
      row = next[e] + __popcll(peers & ((1ull << tid) - 1));
      if (row >= (p.layout == DG_MOE_MASKED ? (e + 1) * p.rows : p.rows)) row = -1;
    }
    rows[tid] = row;
    if (tid < slots) p.row_of[begin + tid] = row;
  }
  if (p.layout == DG_MOE_CONTIGUOUS)
    fill_layout(p, total, first, blockIdx.x * FEW_THREADS + tid, gridDim.x * FEW_THREADS);
  if constexpr (MODE != MOVE_NONE) {
    __syncthreads();
    for (int i = first_item; i < tokens * blocks; i += FEW_THREADS / 16) {
      const int t = i / blocks, b = i - t * blocks;  // the tokens' blocks follow one another
      if (i >= FEW_THREADS / 16) raw = load16(m.x + (size_t)t0 * p.hidden + (size_t)i * QBLOCK + l16 * 8);
      for (int j0 = 0; j0 < k; j0 += 16) {
        const int here = min(k - j0, 16);
        put_block<MODE>(p, m, raw, b, l16, l16 < here ? rows[t * k + j0 + l16] : -1, here);
      }
    }
  }
}

// Rows back to tokens: a thread sums 8 columns of a token over its slots, the
// rows of 8 slots on their way at once. Bound by memory: every row is read
// once. A row of values is spread over workgroups too (`parts` of them), so
// that a few hundred tokens fill the device. 8192 tokens of 8 rows of 7168: 171
// us (6.2 TB/s); 259 tokens: 7.2 us (4.6 TB/s; one row's loads after the other
// and a workgroup a token took 20).
constexpr int COMBINE_THREADS = 256;
constexpr int AHEAD = 8;

__global__ __launch_bounds__(COMBINE_THREADS) void combine_kernel(RouteArgs p, const uint16_t* yp, const float* w,
                                                               uint16_t* y, uint32_t parts, uint32_t items) {
  const int lane = threadIdx.x & 63;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t t = item / parts, c = ((item - t * parts) * blockDim.x + threadIdx.x) * 8;
    const bool inside = c < (uint32_t)p.hidden;
    const int32_t mine = lane < p.top_k ? p.row_of[(size_t)t * p.top_k + lane] : -1;
    const float weight = mine >= 0 ? (w ? w[(size_t)t * p.top_k + lane] : 1.0f) : 0.0f;
    F8 acc = {};
    for (int j0 = 0; j0 < p.top_k; j0 += AHEAD) {
      u32x4 v[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        v[j] = (u32x4){0, 0, 0, 0};
        const int r = __builtin_amdgcn_readlane(mine, j0 + j);  // top_k <= 32: -1 past it
        if (r >= 0 && inside) v[j] = load_stream16(yp + (size_t)r * p.hidden + c);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const float wj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j0 + j));
        const F8 f = unpack8(v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc.v[i] = __builtin_fmaf(wj, f.v[i], acc.v[i]);
      }
    }
    if (inside) store_stream(y + (size_t)t * p.hidden + c, pack8(acc));
  }
}

// Its gradient: a workgroup a token, the token's gradient read once per 8
// slots, their rows on the way at once. Bound by memory (rows read, rows
// written); the sums for the weights' gradients stay in registers. 26500 rows of
// 7168: 152 us (5.7 TB/s).
constexpr int BWD_THREADS = 512;

__global__ __launch_bounds__(BWD_THREADS) void combine_bwd_kernel(RouteArgs p, const uint16_t* dy, const uint16_t* yp,
                                                                  const float* w, uint16_t* dyp, float* dw) {
  __shared__ float scratch[2][BWD_THREADS / 64][AHEAD];
  const size_t t = blockIdx.x, H = p.hidden;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int32_t mine = lane < p.top_k ? p.row_of[t * p.top_k + lane] : -1;
  const float weight = mine >= 0 ? w[t * p.top_k + lane] : 0.0f;
  int turn = 0;
  for (int j0 = 0; j0 < p.top_k; j0 += AHEAD) {
    if (!__ballot(lane >= j0 && lane < j0 + AHEAD && mine >= 0)) {  // no row among these slots
      if (dw && threadIdx.x < AHEAD && j0 + (int)threadIdx.x < p.top_k) dw[t * p.top_k + j0 + threadIdx.x] = 0.0f;
      continue;
    }
    float dot[AHEAD] = {};
    int r[AHEAD];
    float wj[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      r[j] = __builtin_amdgcn_readlane(mine, j0 + j);
      wj[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j0 + j));
    }
    for (size_t c = threadIdx.x * 8; c < H; c += blockDim.x * 8) {
      u32x4 v[AHEAD];
      const u32x4 raw = load_stream16(dy + t * H + c);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        v[j] = (u32x4){0, 0, 0, 0};
        if (r[j] >= 0 && dw) v[j] = load_stream16(yp + (size_t)r[j] * H + c);
      }
      const F8 d = unpack8(raw);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (r[j] < 0) continue;
        const F8 f = unpack8(v[j]);
        F8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o.v[i] = wj[j] * d.v[i];
          dot[j] = __builtin_fmaf(d.v[i], f.v[i], dot[j]);
        }
        store_stream(dyp + (size_t)r[j] * H + c, pack8(o));
      }
    }
    if (!dw) continue;
    float(*s)[AHEAD] = scratch[turn];
    turn ^= 1;  // (blocks of slots that were skipped had no barrier, so they take no turn)
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const float sum = r[j] >= 0 ? wave_sum(dot[j]) : 0.0f;
      if (lane == j) s[wave][j] = sum;
    }
    __syncthreads();
    if (wave == 0 && lane < AHEAD && j0 + lane < p.top_k) {
      float sum = 0.f;
      for (int i = 0; i < waves; ++i) sum += s[i][lane];
      dw[t * p.top_k + j0 + lane] = sum;
    }
  }
}

}  // namespace

// Enough for any number of slots up to `slots` (fewer slots may take more,
// smaller chunks).
long long sort_workspace(int slots, int num_groups) {
  const int chunks = std::min((slots + SORT_THREADS - 1) / SORT_THREADS, MAX_CHUNKS);
  return (long long)std::max(chunks, 1) * num_groups * 4;
}

namespace {

// Whether one launch sorts (and moves), where that beats the passes over chunks.
// Times in us, 64 groups, FP8, first the one launch: ids spread evenly / by a Zipf
// law of exponent 1.2, whose counting meets on few counters.
//   sort alone     4096 slots                4.7 /  7.2 against  6.9 /  7.0
//                  8192                      6.2 / 11.3 against  7.1 /  7.2
//   rows of 256    8192 of 4096 tokens       7.3 / 11.4 against  9.9 /  9.9
//                  16384 of 4096            10.0 / 16.2 against 10.4 / 10.5
//   rows of 4096   16384 of 4096            28.6 / 28.9 against 30.0 / 29.9
//   rows of 7168   8192 of 1024             19.9 / 19.6 against 24.9 / 25.0
//                  16384 of 4096            41.0 / 41.5 against 45.8 / 45.5
// More tokens than that are too many for each workgroup, which moves its own in
// turn: 8192 slots of 8192 tokens of 7168  55.4 / 58.0 against 46.8 / 46.2.
bool one_launch(const RouteArgs& a, bool moves) {
  const int slots = a.tokens * a.top_k;
  if (!moves) return slots <= 4096;
  return a.tokens <= 4096 && slots <= (a.hidden >= 4096 ? FEW_SLOTS : 8192);
}

template <int MODE>
hipError_t launch_one(const RouteArgs& a, const MoveArgs& m, hipStream_t stream) {
  const int each = std::max((a.tokens + FEW_WORKGROUPS - 1) / FEW_WORKGROUPS, 1);
  const int fills = a.layout == DG_MOE_CONTIGUOUS ? std::min((a.rows + FILL_ROWS - 1) / FILL_ROWS, 64) : 1;
  const int grid = (std::max({(a.tokens + each - 1) / each, fills, 1}) + 7) / 8 * 8;
  hipLaunchKernelGGL(few_kernel<MODE>, dim3(grid), dim3(FEW_THREADS), 0, stream, a, m, each);
  return hipGetLastError();
}

hipError_t launch_passes(const RouteArgs& a, hipStream_t stream) {
  const int slots = a.tokens * a.top_k, chunk = chunk_slots(slots), chunks = (slots + chunk - 1) / chunk;
  hipLaunchKernelGGL(count_kernel, dim3(chunks), dim3(SORT_THREADS), 0, stream, a, chunk);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(rank_kernel, dim3(chunks), dim3(SORT_THREADS), 0, stream, a, chunk, chunks);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_move(const RouteArgs& a, const MoveArgs& m, hipStream_t stream) {
  if (a.ids) {
    if (one_launch(a, true)) return launch_one<MODE>(a, m, stream);
    if (hipError_t e = launch_passes(a, stream)) return e;
  }
  const long long groups = (long long)((a.tokens + 7) / 8) * (a.hidden / QBLOCK);
  const int per_xcd = (int)std::min<long long>((groups + DISPATCH_THREADS / 16 - 1) / (DISPATCH_THREADS / 16), 1 << 19);
  hipLaunchKernelGGL(dispatch_kernel<MODE>, dim3(per_xcd * 8), dim3(DISPATCH_THREADS), 0, stream, a, m);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sort(const RouteArgs& a, hipStream_t stream) {
  return one_launch(a, false) ? launch_one<MOVE_NONE>(a, MoveArgs{}, stream) : launch_passes(a, stream);
}

hipError_t launch_dispatch(const RouteArgs& a, const void* x, void* xp, hipStream_t stream) {
  const MoveArgs m{static_cast<const uint16_t*>(x), static_cast<uint8_t*>(xp), nullptr};
  return launch_move<MOVE_BF16>(a, m, stream);
}

hipError_t launch_dispatch_fp8(const RouteArgs& a, const void* x, void* q, float* sfa, bool ue8m0,
                               hipStream_t stream) {
  const MoveArgs m{static_cast<const uint16_t*>(x), static_cast<uint8_t*>(q), sfa};
  return ue8m0 ? launch_move<MOVE_FP8_E8>(a, m, stream) : launch_move<MOVE_FP8>(a, m, stream);
}

namespace {

// Threads (a multiple of 64 up to `most`) of workgroups that share `pieces`
// of work: the fewest idle ones, and of those the most threads.
int even_threads(int pieces, int most) {
  int best = 64;
  auto idle = [&](int n) { return (pieces + n - 1) / n * n - pieces; };
  for (int n = 128; n <= most; n += 64)
    if (idle(n) <= idle(best)) best = n;
  return best;
}

}  // namespace

hipError_t launch_combine(const RouteArgs& a, const void* yp, const float* w, void* y, hipStream_t stream) {
  const int threads = even_threads(a.hidden / 8, COMBINE_THREADS);
  const uint32_t parts = (a.hidden / 8 + threads - 1) / threads;
  const uint32_t items = parts * (uint32_t)a.tokens;  // below 2^31: tokens take less than 2^40 bytes
  hipLaunchKernelGGL(combine_kernel, dim3(std::min(items, 1u << 22)), dim3(threads), 0, stream, a,
                     static_cast<const uint16_t*>(yp), w, static_cast<uint16_t*>(y), parts, items);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const RouteArgs& a, const void* dy, const void* yp, const float* w, void* dyp,
                              float* dw, hipStream_t stream) {
  hipLaunchKernelGGL(combine_bwd_kernel, dim3(a.tokens), dim3(pass_threads(a.hidden / 8, BWD_THREADS)), 0, stream, a,
                     static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(yp), w,
                     static_cast<uint16_t*>(dyp), dw);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace dg
