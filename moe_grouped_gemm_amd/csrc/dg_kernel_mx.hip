// FP4 NT GEMM with one E8M0 scale per 32 values of either operand (MXFP4) and
// BF16 output, dense and M-grouped, for gfx950 (MI355X):
//
//   D[m][n] = bf16( sum_k e2m1(A[m][k]) 2^(ea[m][k/32] - 127) * e2m1(B[n][k]) 2^(eb[n][k/32] - 127) )
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes packed E2M1 for both operands: lane
// group g = lane / 16 holds 32 successive values of row lane % 16 (16 bytes, even
// k in the low nibble), which are one scale block, and applies the block's two
// scales itself: a byte of the lane's scale register, the same byte in all lanes.
// Its float32 accumulator holds the sums: no step of the kernel's own follows the
// products but the one rounding to BF16.
//
// Which 32 values a group holds is free as long as both operands hold the same. Of a
// step's 256 the j-th of two MFMAs (j = 0, 1) takes blocks 2g + j: a group's two
// blocks have two successive bytes of one scale word, so that a byte permutation puts
// the scales of two 16-row bands and both MFMAs into one register: 6 of them and 3
// reads a step, the words lying in LDS with a row of four bands side by side. (With the
// j-th MFMA on blocks 4j + g every lane would need another byte of its word: a
// transpose between lanes, 36 instructions a step, that cost 8% of the time.)
//
// Two kernels: for few tiles see the second. The first is persistent over 256 x 256
// tiles (or, for fewer of them, 128 x 256), a 128 x 64 part of one a wave; a K step is 256 values, 128-byte rows of either
// operand, in one of two LDS stages that direct-to-LDS loads fill a step and a half
// ahead (see the K loop). Two stages of 68 KB are what LDS holds; smaller tiles read
// more of either operand for a product, and four waves of 128 x 128 (a third fewer LDS
// reads) took 6% more.
//
// What bounds it (16384 x 4096 x 7168 in 215 us, 4.48 PFLOP/s): matrix cores and
// LDS reads alone take 147 us (6.5 PFLOP/s; a loop of these MFMAs alone, with operands
// of random bits, 7.3: they draw the power), a stream of operands that all hit the L1
// 25 us more, from L2 another 26 (its misses 5 of them), the stores 18. 4096 x 7168 x
// 2048 (37 to 40 us by the inputs' power) is two rounds of 224 tiles of 256 possible and
// 10 us of stores. With few rows (16 groups of up to 32 rows, 7168 x 2048, 28 us a call)
// reading B bounds it, at 4.4 TB/s.

#include <algorithm>

#include "dg_device.h"

namespace dg {
namespace mx {

// A workgroup's tile: BM x 256, a wave 128 x 64 of it.
template <int BM_>
struct Cfg {
  static constexpr int BM = BM_, BN = 256, SLOTS = BM / 128;
  static constexpr int WAVES_N = 4, NW = BM / 32, THREADS = NW * 64;
  static constexpr int WM = 128, WN = 64, MT = WM / 16, NT = WN / 16;
};
using Big = Cfg<256>;
using Half = Cfg<128>;
constexpr int STEP_BLOCKS = 2;  // 128-value blocks of K a step: 128-byte rows
// LDS of a stage, in two buffers that are refilled at different times (see the K loop):
// HIGH the later halves of the wave rows' A rows (64 .. 127 of each 128), LOW all else.
enum { LOW = 0, HIGH = 1 };
template <class C>
constexpr int A_HALF = C::BM / 2 * ROW_BYTES;
template <class C>
constexpr int SA_OFF = A_HALF<C> + C::BN * ROW_BYTES;  // [128 values of the step][BM / 64][16][4] LHS scale words: row 64 i + 16 j + r at [i][r][j]
template <class C>
constexpr int SB_OFF = SA_OFF<C> + STEP_BLOCKS * C::BM * 4;
template <class C>
constexpr int LOW_BYTES = SB_OFF<C> + STEP_BLOCKS * C::BN * 4;

// The kernel for few tiles (see there).
struct Few {
  static constexpr int BM = 64, BN = 64, SLOTS = 1;
  static constexpr int NW = 4, THREADS = NW * 64;
};

}  // namespace mx

template <int BM>
constexpr int A_PACK_SHIFT<mx::Cfg<BM>> = 1;
template <>
constexpr int A_PACK_SHIFT<mx::Few> = 1;
template <int BM>
constexpr bool FP8_RHS<mx::Cfg<BM>> = false;
template <>
constexpr bool FP8_RHS<mx::Few> = false;

namespace mx {

// An LDS buffer for each stage and half, and its byte address.
template <class C, int S, int PART>
__device__ __forceinline__ uint8_t* stage_buf() {
  __shared__ __attribute__((aligned(1024))) uint8_t buf[PART == LOW ? LOW_BYTES<C> : A_HALF<C>];
  return buf;
}
template <class C, int S, int PART>
__device__ __forceinline__ uint32_t stage_addr() {
  return (uint32_t)(uintptr_t)(lds_void*)stage_buf<C, S, PART>();
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 4, voff, 0, 0, 0);
}

// This lane's byte offsets within a tile: of its A and B loads (the j-th adds 8 NW j
// rows) and of its scale words.
struct LaneOffsets {
  uint32_t ab, ab_step, sa, sb;
};

template <class C>
__device__ __forceinline__ LaneOffsets lane_offsets(int k, int wave, int lane) {
  LaneOffsets o;
  const int row0 = wave * 8 + (lane >> 3);
  // Of the row's eight 16-byte blocks 2g + j lies where lds_offset() has chunk g + 4j.
  const int chunk = (lane & 7) ^ ((row0 >> 1) & 7);  // the same for every j
  o.ab = (uint32_t)row0 * ((uint32_t)k / 2) + (uint32_t)((chunk & 3) * 2 + (chunk >> 2)) * 16u;
  o.ab_step = 8u * C::NW * ((uint32_t)k / 2);
  const int word = (lane & 3) * 16 + (lane >> 2);
  o.sa = (uint32_t)(64 * (wave % (C::BM / 64)) + word) * 4u;
  o.sb = (uint32_t)(64 * (wave & 3) + word) * 4u;
  return o;
}

// Where a tile's operands start (the group's B and its scales are located from the
// group index), and the byte extents past which its rows read as zero.
struct TileSrc {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  uint32_t a_rows, b_rows;
};

template <class C>
__device__ __forceinline__ TileSrc tile_src(const GemmArgs& p, const TileRef& tr) {
  static_assert(!FP8_RHS<C> && A_PACK_SHIFT<C> == 1, "both operands are packed");
  TileSrc s;
  const size_t row = (size_t)p.k / 2;
  s.a_rows = uniform_int(min(max(tr.load_rows - tr.m0, 0), C::BM));
  s.b_rows = uniform_int(min(p.n - tr.n0, C::BN));
  s.a = uniform_ptr(tr.a + (size_t)tr.m0 * row);
  s.sa = uniform_ptr(tr.sfa + tr.m0);
  s.b = uniform_ptr(p.b + ((size_t)tr.group * p.n + tr.n0) * row);
  s.sb = uniform_ptr(p.sfb + (size_t)tr.group * (p.k / BK) * p.ld_sfb + tr.n0);
  return s;
}

// Buffer descriptors of one step of one tile. Rows past the matrix read as zero. So does
// everything of an odd last block's second half: the scale words by their
// descriptors, and codes that are other rows' (no code is infinite or NaN) come to
// nothing under two scales of 2^-127.
template <class C>
struct StageSrc {
  static constexpr int SB_LOADS = 8 / C::NW;  // of 64 words each
  __amdgpu_buffer_rsrc_t a, b, sa, sb[SB_LOADS];
};

template <class C>
__device__ __forceinline__ StageSrc<C> stage_src(const GemmArgs& p, const TileSrc& t, int step, int wave) {
  StageSrc<C> r;
  const uint32_t row = (uint32_t)p.k / 2, skip = (uint32_t)step * ROW_BYTES;
  auto words = [&](const float* w, int block, int ld, uint32_t rows) {  // `block` of the step's
    const int blk = step * STEP_BLOCKS + block;
    return buffer_rsrc(w + (size_t)blk * ld, blk < p.k / BK ? rows * 4u : 0);
  };
  r.a = buffer_rsrc(t.a + skip, t.a_rows ? t.a_rows * row - skip : 0);
  r.b = buffer_rsrc(t.b + skip, t.b_rows * row - skip);
  r.sa = words(t.sa, wave / (C::BM / 64), p.ld_sfa, t.a_rows);
#pragma unroll
  for (int i = 0; i < r.SB_LOADS; ++i) r.sb[i] = words(t.sb, (i * C::NW + wave) >> 2, p.ld_sfb, t.b_rows);
  return r;
}

// Descriptors of the step `ahead` steps after step 0 of the current tile: a step of
// this tile, of the next one, or (with a single step per tile) of the one after.
// With no such tile the window's entries repeat the previous one and the loads fetch
// a step nobody reads.
template <class C>
__device__ __forceinline__ StageSrc<C> refill_src(const GemmArgs& p, const TileSrc& t0, const TileSrc& t1,
                                               const TileSrc& t2, int ahead, int steps, int wave) {
  const bool in0 = ahead < steps, in1 = ahead < 2 * steps;
  // Field by field (a select between references would put the tiles in memory).
  TileSrc t;
  t.a = in0 ? t0.a : (in1 ? t1.a : t2.a);
  t.b = in0 ? t0.b : (in1 ? t1.b : t2.b);
  t.sa = in0 ? t0.sa : (in1 ? t1.sa : t2.sa);
  t.sb = in0 ? t0.sb : (in1 ? t1.sb : t2.sb);
  t.a_rows = in0 ? t0.a_rows : (in1 ? t1.a_rows : t2.a_rows);
  t.b_rows = in0 ? t0.b_rows : (in1 ? t1.b_rows : t2.b_rows);
  return stage_src<C>(p, t, in0 ? ahead : (in1 ? ahead - steps : ahead - 2 * steps), wave);
}

// The loads of one step into stage S: 0 and 1 the B tile, 2 the LOW half of the A tile,
// 3 the scale words, 4 the HIGH half of the A tile. How many of a wave each takes:
template <class C, int PART>
constexpr int PART_LOADS = PART < 2 ? 16 / C::NW : PART == 3 ? 1 + StageSrc<C>::SB_LOADS : 2;
template <class C>
constexpr int LOW_LOADS = 2 * PART_LOADS<C, 0> + PART_LOADS<C, 2> + PART_LOADS<C, 3>;
constexpr int HIGH_LOADS = 2;
template <class C, int S, int PART>
__device__ __forceinline__ void issue_part(const StageSrc<C>& r, int wave, const LaneOffsets& lo) {
  const uint32_t st = stage_addr<C, S, PART == 4 ? HIGH : LOW>();
  if constexpr (PART == 3) {
    dma4(r.sa, lo.sa, st + SA_OFF<C> + wave * 256);
#pragma unroll
    for (int i = 0; i < r.SB_LOADS; ++i) dma4(r.sb[i], lo.sb, st + SB_OFF<C> + (i * C::NW + wave) * 256);
  } else {
    constexpr int ROUNDS = 8 / C::NW;  // that 64 rows take
#pragma unroll
    for (int i = 0; i < PART_LOADS<C, PART>; ++i) {
      // Which 8 NW rows of the tile, and of its place in LDS.
      const int slot = PART < 2 ? PART * PART_LOADS<C, PART> + i : i;
      const int j = PART < 2 ? slot : i / ROUNDS * 2 * ROUNDS + i % ROUNDS + (PART == 4) * ROUNDS;
      dma16(PART < 2 ? r.b : r.a, lo.ab + j * lo.ab_step, st + (PART < 2 ? A_HALF<C> : 0) + (slot * C::NW + wave) * 1024);
    }
  }
}

// A lane's LDS byte offsets within a stage, fixed for the kernel (a 16-row band adds
// 2048 bytes; see lds_offset() for the swizzle).
struct LdsOffsets {
  uint32_t a0, a1, b0, b1;  // what the lane holds for the two MFMAs, of the wave's first band or columns
  uint32_t sa, sb;          // its scale words of four bands or column blocks
  uint32_t pick;            // byte selector: of two words, the two bytes of each that the lane needs
};

template <class C>
__device__ __forceinline__ LdsOffsets lds_offsets(int wm0, int wn0, int lane) {
  LdsOffsets o;
  const int r = lane & 15, g = lane >> 4;
  const uint32_t c0 = (uint32_t)lds_offset(r, g), c1 = (uint32_t)lds_offset(r, g + 4);
  o.a0 = (uint32_t)wm0 / 2 * ROW_BYTES + c0;
  o.a1 = (uint32_t)wm0 / 2 * ROW_BYTES + c1;
  o.b0 = A_HALF<C> + (uint32_t)wn0 * ROW_BYTES + c0;
  o.b1 = A_HALF<C> + (uint32_t)wn0 * ROW_BYTES + c1;
  o.sa = SA_OFF<C> + (uint32_t)((g >> 1) * C::BM * 4 + wm0 * 4 + r * 16);
  o.sb = SB_OFF<C> + (uint32_t)((g >> 1) * C::BN * 4 + wn0 * 4 + r * 16);
  o.pick = (g & 1) ? 0x07060302u : 0x05040100u;
  return o;
}

// A 16-row fragment for both MFMAs of a step.
struct Frag {
  i32x4 h[2];
};
template <class C, int S, int PART = LOW>
__device__ __forceinline__ Frag frag_at(uint32_t off0, uint32_t off1, int band) {
  const uint8_t* st = stage_buf<C, S, PART>();
  Frag f;
  f.h[0] = *reinterpret_cast<const i32x4*>(st + off0 + band * 16 * ROW_BYTES);
  f.h[1] = *reinterpret_cast<const i32x4*>(st + off1 + band * 16 * ROW_BYTES);
  return f;
}
template <class C, int S, int BAND>
__device__ __forceinline__ Frag band_at(const LdsOffsets& lds) {
  return frag_at<C, S, BAND / 4>(lds.a0, lds.a1, BAND % 4);
}
__device__ __forceinline__ i32x8 operand(const i32x4& v) { return (i32x8){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The scales of the wave's bands and column blocks, two of them a register: byte
// 2 (i % 2) + j of register i / 2 for the j-th MFMA.
struct Scales {
  int a[Big::MT / 2], b[Big::NT / 2];
};
// The scales of four bands or column blocks, from index 2 I of `to`.
template <class C, int S, int I, int N>
__device__ __forceinline__ void scales_at(int (&to)[N], uint32_t off, uint32_t pick) {
  const i32x4 w = *reinterpret_cast<const i32x4*>(stage_buf<C, S, LOW>() + off + I * 256);
  to[2 * I] = __builtin_amdgcn_perm(w[1], w[0], pick);
  to[2 * I + 1] = __builtin_amdgcn_perm(w[3], w[2], pick);
}

template <int MT, int NT, int H>
__device__ __forceinline__ f32x4 mfma(const Frag& b, const Frag& a, const f32x4& c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.h[H]), operand(a.h[H]), c, 4, 4, 2 * (NT & 1) + H,
                                                          sb, 2 * (MT & 1) + H, sa);
}

// Writes 16 rows of 64 columns as BF16 (round to nearest even), the rows of `valid` only;
// `rows` is the first row's first column. A lane has 4 columns of a row of each 16-column
// block; exchanges between lane halves, quarters and halves of quarters give it 8 of a
// row's 64, so that each store covers whole 128-byte segments of 8 rows. (Without the
// last exchange, 64 bytes of 16 rows a store, the masked decode took 1 to 2% more.)
__device__ __forceinline__ void store_band(uint16_t* rows, int n, uint32_t valid, const f32x4 (&v)[4], int lane) {
  const int r = lane & 15, q = lane >> 4;
  i32x4 w[2];  // columns 32 np + 8 q .. + 7 of row r
#pragma unroll
  for (int np = 0; np < 2; ++np)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // Lanes of quarter q hold columns 4 q + 2 i of either block. The lanes' upper
      // half's first block against the lower half's second, then odd quarters' against
      // even ones': quarter q has columns 8 q .. 8 q + 7 of the 32.
      const f32x4 &x = v[2 * np], &y = v[2 * np + 1];
      const auto h = __builtin_amdgcn_permlane32_swap(pack_bf16x2(x[2 * i], x[2 * i + 1]),
                                                      pack_bf16x2(y[2 * i], y[2 * i + 1]), false, false);
      const auto t = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
      w[np][i] = (int)t[0];
      w[np][2 + i] = (int)t[1];
    }
  // The second 32 columns of rows 0 .. 7 against the first of rows 8 .. 15 (a rotation of
  // each 16 lanes by 8, written to 8 of them).
  i32x4 out[2];  // columns 32 (r / 8) + 8 q .. + 7 of rows r % 8 and 8 + r % 8
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[0][i] = __builtin_amdgcn_update_dpp(w[0][i], w[1][i], 0x128, 0xF, 0xC, false);
    out[1][i] = __builtin_amdgcn_update_dpp(w[1][i], w[0][i], 0x128, 0xF, 0x3, false);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = (r & 7) + 8 * half;
    // Past the caches' reach: the operands stay there (4096 x 7168 x 2048: 40 us, with
    // plain stores 42; 16 masked groups of up to 256 x 7168 x 2048 43 and 46).
    if ((valid >> row) & 1)
      __builtin_nontemporal_store(out[half], (global_i32x4*)(rows + (size_t)row * n + 32 * (r >> 3) + 8 * q));
  }
}

// A wave's finished 128 x 64 sub-tile.
template <class C, int KIND>
__device__ __forceinline__ void store_tile(const GemmArgs& p, const TileRef& cur, const RowMask& cm,
                                           const f32x4 (&acc)[C::MT][C::NT], int wm0, int wn0, int lane) {
  static_assert(C::NT == 4, "a band of 64 columns");
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) {
    const uint32_t valid = band_rows<C, KIND>(cur, cm, wm0, mt);
    if (valid != 0)
      store_band(cur.d + (size_t)(cur.m0 + wm0 + mt * 16) * p.n + cur.n0 + wn0, p.n, valid, acc[mt], lane);
  }
}

// The K loop of one tile; its first step reads stage PHASE. Step i of the global
// sequence of steps reads stage s = i % 2, and issues the loads of step i + 2 into it as
// its parts fall free:
//   entry:     the first step's first operands are read (they were complete before the
//              last barrier);
//   bands 0-1: the A fragment two bands ahead from LOW, 8 MFMAs of the band (4 column
//              blocks, 2 halves of K);
//   barrier:   after it no wave reads LOW of stage s any more (its fragments of B, the
//              scales and bands 2 and 3 are in registers), and every wave's loads of HIGH
//              of stage s have landed;
//   bands 2-5: the same from HIGH; a quarter of LOW's refill is issued with each;
//   barrier:   after it no wave reads HIGH of stage s any more, and every wave's loads of
//              step i + 1 into LOW have landed;
//   bands 6-7: column block by column block, so that a B fragment is read again for step
//              i + 1 as soon as its last MFMA of step i has issued, then the next step's
//              first A fragments and its scales; HIGH's refill is issued.
// So every load has a step and a half to land. (One barrier a step, at band 6, gave it
// 0.6 to 1 step, and took 3.6% more for 16384 x 4096 x 7168.)
// Only bands below NB are computed (the rows of the others are not stored).
template <class C, int KIND, int PHASE, int NB>
__device__ __forceinline__ void mainloop(const GemmArgs& p, const TileSrc& t0, const TileSrc& t1, const TileSrc& t2,
                                         f32x4 (&acc)[C::MT][C::NT], bool on, int wave, int lane,
                                         const LdsOffsets& lds, const LaneOffsets& lo, const RowGroups& nrg, int ngroup,
                                         RowMask& nmask) {
  static_assert(NB == C::MT || (NB >= 2 && NB <= 6), "a partial copy computes bands 0 .. NB-1 before the barrier");
  // The next tile's row mask (contiguous layout), after a barrier: see RowGroups.
  auto next_rows = [&]() {
    if constexpr (KIND == KIND_CONTIGUOUS) {
      int e = nrg.even, o = nrg.odd;
      asm volatile("" : "+v"(e), "+v"(o));  // keeps the compare (and the wait for the loads) here
      nmask = row_mask(RowGroups{e, o}, ngroup);
    }
  };
  const int steps = (p.k / BK + STEP_BLOCKS - 1) / STEP_BLOCKS;
  Frag af[4], bf[C::NT];  // A ring: band mt's fragment in slot mt % 4
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) bf[nt] = frag_at<C, PHASE>(lds.b0, lds.b1, nt);
  af[0] = band_at<C, PHASE, 0>(lds);
  af[1] = band_at<C, PHASE, 1>(lds);
  Scales scales;
  scales_at<C, PHASE, 0>(scales.b, lds.sb, lds.pick);
  scales_at<C, PHASE, 0>(scales.a, lds.sa, lds.pick);
  scales_at<C, PHASE, 1>(scales.a, lds.sa, lds.pick);
  for (int i0 = 0; i0 < steps; i0 += 2) {
    static_for<0, 2>([&](auto si) {
      constexpr int s = (decltype(si)::value + PHASE) % 2, sn = 1 - s;
      const int i = i0 + decltype(si)::value;
      if (i >= steps) return;
      // The refills are issued unconditionally (past the last tile they load a step nobody
      // reads): a branch here would make the compiler wait for them before reading the
      // current stage.
      const StageSrc<C> r2 = refill_src<C>(p, t0, t1, t2, i + 2, steps, wave);
      if (!on) {
        wait_vmcnt<LOW_LOADS<C> + HIGH_LOADS>();
        wait_lgkmcnt_0();
        barrier();
        issue_part<C, s, 0>(r2, wave, lo);
        issue_part<C, s, 1>(r2, wave, lo);
        issue_part<C, s, 2>(r2, wave, lo);
        issue_part<C, s, 3>(r2, wave, lo);
        wait_vmcnt<LOW_LOADS<C> + HIGH_LOADS>();
        barrier();
        next_rows();
        issue_part<C, s, 4>(r2, wave, lo);
        return;
      }
      static_for<0, 6>([&](auto MT) {
        constexpr int mt = decltype(MT)::value;
        if constexpr (mt == 2) {
          wait_lgkmcnt_0();
          wait_vmcnt<LOW_LOADS<C> + HIGH_LOADS>();  // all but the last refills of LOW and HIGH
          barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (mt + 2 < NB) af[(mt + 2) % 4] = band_at<C, s, mt + 2>(lds);
        if constexpr (mt >= 2) issue_part<C, s, mt - 2>(r2, wave, lo);
        if constexpr (mt < NB) {
          static_for<0, 2 * C::NT>([&](auto I) {
            constexpr int h = decltype(I)::value / C::NT, nt = decltype(I)::value % C::NT;
            acc[mt][nt] = mfma<mt, nt, h>(bf[nt], af[mt % 4], acc[mt][nt], scales.b[nt / 2], scales.a[mt / 2]);
          });
          // The reads two bands ahead and this band's share of the refill first.
          if constexpr (mt + 2 < NB) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // DS reads
          if constexpr (mt >= 2) __builtin_amdgcn_sched_group_barrier(0x020, PART_LOADS<C, mt - 2>, 0);  // VMEM loads
          __builtin_amdgcn_sched_group_barrier(0x008, 2 * C::NT, 0);  // MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<0, C::NT>([&](auto NT) {
        constexpr int nt = decltype(NT)::value;
        if constexpr (NB == C::MT) {
          acc[6][nt] = mfma<6, nt, 0>(bf[nt], af[2], acc[6][nt], scales.b[nt / 2], scales.a[6 / 2]);
          acc[7][nt] = mfma<7, nt, 0>(bf[nt], af[3], acc[7][nt], scales.b[nt / 2], scales.a[7 / 2]);
          acc[6][nt] = mfma<6, nt, 1>(bf[nt], af[2], acc[6][nt], scales.b[nt / 2], scales.a[6 / 2]);
          acc[7][nt] = mfma<7, nt, 1>(bf[nt], af[3], acc[7][nt], scales.b[nt / 2], scales.a[7 / 2]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (nt == 0) {
          wait_lgkmcnt_0();
          wait_vmcnt<LOW_LOADS<C> + HIGH_LOADS>();  // the same
          barrier();
          next_rows();
          __builtin_amdgcn_sched_barrier(0);
          issue_part<C, s, 4>(r2, wave, lo);
        }
        // The next step's operands (past a tile's last step: the next tile's first, which
        // its entry reads again).
        bf[nt] = frag_at<C, sn>(lds.b0, lds.b1, nt);
        if constexpr (nt == 1) af[0] = band_at<C, sn, 0>(lds);
        if constexpr (nt == 3) {  // bands 6 and 7 are done
          af[1] = band_at<C, sn, 1>(lds);
          scales_at<C, sn, 0>(scales.b, lds.sb, lds.pick);
          scales_at<C, sn, 0>(scales.a, lds.sa, lds.pick);
          scales_at<C, sn, 1>(scales.a, lds.sa, lds.pick);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }
}

// A wave whose valid rows lie in its first HALF_BANDS bands runs a copy of the K loop
// without the other bands' MFMAs (their rows are never stored). 32 groups of up to 64
// rows, 4096 x 7168: 90 us, without the copy 96; 16 groups of up to 256 rows, 7168 x
// 2048: 43 with either.
constexpr int HALF_BANDS = 4;

template <class C, int KIND>
__global__ void __launch_bounds__(C::THREADS, 1) fp4_gemm_nt_kernel(GemmArgs p) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / C::WAVES_N) * C::WM;
  const int wn0 = (wave % C::WAVES_N) * C::WN;
  const int steps = (p.k / BK + STEP_BLOCKS - 1) / STEP_BLOCKS;

  int num_tiles = p.num_tiles;
  [[maybe_unused]] int* s_prefix = nullptr;
  if constexpr (counts_on_device(KIND)) {
    s_prefix = group_table<C, KIND>(p, tid);
    num_tiles = s_prefix[p.num_groups];
  }

  // Each XCD takes a contiguous range of tiles per round.
  const int grid = gridDim.x;
  int rank = blockIdx.x;
  if ((grid & 7) == 0) rank = (blockIdx.x & 7) * (grid >> 3) + (blockIdx.x >> 3);

  // A window of three tiles: the current one and the next two (refills run two steps
  // ahead, which reaches the tile after next when a tile has a single step). Missing
  // tiles repeat the previous window entry.
  int t = rank;
  TileRef cur = next_active<C, KIND>(p, t, grid, num_tiles, s_prefix);
  if (!cur.active) return;
  int t1 = t + grid;
  TileRef nxt = next_active<C, KIND>(p, t1, grid, num_tiles, s_prefix);
  int t2 = t1 + grid;
  TileRef nx2;
  nx2.active = false;
  if (nxt.active) nx2 = next_active<C, KIND>(p, t2, grid, num_tiles, s_prefix);
  const LaneOffsets lo = lane_offsets<C>(p.k, wave, lane);
  const LdsOffsets lds = lds_offsets<C>(wm0, wn0, lane);
  TileSrc c0 = tile_src<C>(p, cur);
  TileSrc c1 = nxt.active ? tile_src<C>(p, nxt) : c0;
  TileSrc c2 = nx2.active ? tile_src<C>(p, nx2) : c1;

  // The first tile's row groups (contiguous layout) are loaded before the prologue's
  // loads, so that waiting for them never waits for those.
  [[maybe_unused]] RowGroups crg{-1, -1};
  if constexpr (KIND == KIND_CONTIGUOUS) crg = load_row_groups<C>(p, cur, wm0, lane);

  // Steps 0 and 1; of step 0 LOW must have landed for every wave before it is read.
  {
    const StageSrc<C> r0 = refill_src<C>(p, c0, c1, c2, 0, steps, wave);
    const StageSrc<C> r1 = refill_src<C>(p, c0, c1, c2, 1, steps, wave);
    static_for<0, 5>([&](auto I) { issue_part<C, 0, decltype(I)::value>(r0, wave, lo); });
    static_for<0, 5>([&](auto I) { issue_part<C, 1, decltype(I)::value>(r1, wave, lo); });
    wait_vmcnt<LOW_LOADS<C> + 2 * HIGH_LOADS>();
    barrier();
  }
  int phase = 0;

  RowMask cmask{0, 0}, nmask{0, 0};
  if constexpr (KIND == KIND_CONTIGUOUS) cmask = row_mask(crg, cur.group);

  while (cur.active) {
    bool any_row;
    if constexpr (KIND == KIND_CONTIGUOUS) any_row = (cmask.even | cmask.odd) != 0;
    else any_row = cur.valid_rows > cur.m0 + wm0;
    const bool on = any_row && cur.n0 + wn0 < p.n;
    int bands = C::MT;
    if constexpr (counts_on_device(KIND))
      bands = uniform_int(min(max((cur.valid_rows - cur.m0 - wm0 + 15) / 16, 0), C::MT));
    RowGroups nrg{-1, -1};
    if constexpr (KIND == KIND_CONTIGUOUS) nrg = load_row_groups<C>(p, nxt, wm0, lane);
    f32x4 acc[C::MT][C::NT];
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) acc[mt][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};

    if (counts_on_device(KIND) && bands <= HALF_BANDS) {
      if (phase == 0) mainloop<C, KIND, 0, HALF_BANDS>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
      else mainloop<C, KIND, 1, HALF_BANDS>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
    } else {
      if (phase == 0) mainloop<C, KIND, 0, C::MT>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
      else mainloop<C, KIND, 1, C::MT>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
    }
    phase = (phase + steps) & 1;

    if (on) store_tile<C, KIND>(p, cur, cmask, acc, wm0, wn0, lane);
    // Slide the window.
    cmask = nmask;
    cur = nxt;
    c0 = c1;
    nxt = nx2;
    c1 = c2;
    if (nx2.active) {
      t2 += grid;
      nx2 = next_active<C, KIND>(p, t2, grid, num_tiles, s_prefix);
    }
    c2 = nx2.active ? tile_src<C>(p, nx2) : c1;
  }
  // The last refills loaded steps nobody reads; no wave may end while such a load can
  // still write its LDS.
  wait_vmcnt_0();
}

// ---------------------------------------------------------------------------
// Few tiles
// ---------------------------------------------------------------------------

// 64 x 64 tiles, the K of each shared by a workgroup's four waves, step by step in
// turn: each wave loads both operands of its steps into a ring of its own, one step ahead,
// and needs no barrier; at a tile's end their sums meet in LDS, added in order. Sixteen
// times the tiles and a fourth of the steps of the kernel above, and four times its
// operand traffic.
constexpr int FEW_SA = (Few::BM + Few::BN) * ROW_BYTES;  // LDS of a step: A, B, the words of A [block][r][band] and B
constexpr int FEW_SB = FEW_SA + STEP_BLOCKS * Few::BM * 4;
constexpr int FEW_STEP = FEW_SB + STEP_BLOCKS * Few::BN * 4;
constexpr int FEW_LOADS = 2 * 8 + 2 * STEP_BLOCKS;
static_assert(2 * FEW_STEP >= 4 * 4 * 64 * 16, "a wave's sums in its ring's place");

// Tile t of the contiguous layout: a 128-row block belongs to its first row's group.
__device__ __forceinline__ TileRef few_contiguous_tile(const GemmArgs& p, int t) {
  TileRef tr;
  int mb, nb;
  raster(t, p.m_blocks, p.n_blocks, 4, mb, nb);
  tr.m0 = uniform_int(mb * Few::BM);
  tr.n0 = uniform_int(nb * Few::BN);
  tr.load_rows = tr.valid_rows = p.m;
  tr.a = p.a;
  tr.sfa = p.sfa;
  tr.d = p.d;
  tr.group = aux_scalar(p.aux, tr.m0 & ~127);
  tr.active = tr.group >= 0 && tr.group < p.num_groups;
  return tr;
}

template <int KIND>
__global__ void __launch_bounds__(Few::THREADS, 1) fp4_gemm_few_kernel(GemmArgs p) {
  static_assert(!FP8_RHS<Few> && A_PACK_SHIFT<Few> == 1, "both operands are packed");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Few::NW * 2 * FEW_STEP];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k_blocks = p.k / BK, steps = (k_blocks + STEP_BLOCKS - 1) / STEP_BLOCKS;
  const int mine = max((steps - wave + Few::NW - 1) / Few::NW, 0);
  int num_tiles = p.num_tiles;
  [[maybe_unused]] int* s_prefix = nullptr;
  if constexpr (counts_on_device(KIND)) {
    s_prefix = group_table<Few, KIND>(p, tid);
    num_tiles = s_prefix[p.num_groups];
  }
  uint8_t* const ring = lds + wave * 2 * FEW_STEP;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void*)ring, row = (uint32_t)p.k / 2;
  // The lane's 16 bytes of each 8 rows of a load, rows 8 j .. (see lane_offsets()).
  uint32_t load_at[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row0 = 8 * j + (lane >> 3), chunk = (lane & 7) ^ ((row0 >> 1) & 7);
    load_at[j] = (uint32_t)(lane >> 3) * row + (uint32_t)((chunk & 3) * 2 + (chunk >> 2)) * 16u;
  }
  const uint32_t word_row = (uint32_t)((lane & 3) * 16 + (lane >> 2));
  const uint32_t c0 = (uint32_t)lds_offset(r, g), c1 = (uint32_t)lds_offset(r, g + 4);
  const uint32_t words_at = (uint32_t)((g >> 1) * 256 + r * 16), pick = (g & 1) ? 0x07060302u : 0x05040100u;

  for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
    TileRef cur;
    [[maybe_unused]] int id = 0;
    if constexpr (KIND == KIND_CONTIGUOUS) {
      cur = few_contiguous_tile(p, t);
      if (!cur.active) continue;
      id = p.aux[cur.m0 + lane];
    } else {
      int at = t;
      cur = next_active<Few, KIND>(p, at, gridDim.x, num_tiles, s_prefix);  // (every tile is active)
    }
    const int rows = uniform_int(min(cur.load_rows - cur.m0, Few::BM)), bands = (rows + 15) / 16;
    const __amdgpu_buffer_rsrc_t a = buffer_rsrc(cur.a + (size_t)cur.m0 * row, (uint32_t)rows * row);
    const __amdgpu_buffer_rsrc_t b = buffer_rsrc(p.b + ((size_t)cur.group * p.n + cur.n0) * row, Few::BN * row);
    // The group's words. Those of rows past the tile's are other rows', and reach no row
    // that is stored; a second block past the last reads as zero (see stage_src()).
    const uint32_t sa_bytes = (uint32_t)k_blocks * p.ld_sfa * 4, sb_bytes = (uint32_t)k_blocks * p.ld_sfb * 4;
    const float* const sfa = KIND == KIND_MASKED ? cur.sfa : p.sfa;
    const __amdgpu_buffer_rsrc_t sa = buffer_rsrc(sfa, sa_bytes);
    const __amdgpu_buffer_rsrc_t sb = buffer_rsrc(p.sfb + (size_t)cur.group * k_blocks * p.ld_sfb, sb_bytes);
    const uint32_t sa_at = ((uint32_t)(cur.sfa - sfa) + cur.m0 + word_row) * 4, sb_at = (cur.n0 + word_row) * 4;
    auto load = [&](int i) {
      const int step = i * Few::NW + wave;
      const uint32_t st = base + (i & 1) * FEW_STEP, skip = (uint32_t)step * ROW_BYTES;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(a, lds_dest(st + j * 1024), 16, load_at[j & 1] + 8 * j * row, skip, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds_dest(st + Few::BM * ROW_BYTES + j * 1024), 16,
                                                 load_at[j & 1] + 8 * j * row, skip, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < STEP_BLOCKS; ++j) {
        const uint32_t blk = (uint32_t)(step * STEP_BLOCKS + j);
        dma4(sa, sa_at + blk * p.ld_sfa * 4, st + FEW_SA + j * 256);
        dma4(sb, sb_at + blk * p.ld_sfb * 4, st + FEW_SB + j * 256);
      }
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) acc[mt][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (mine > 0) load(0);
    for (int i = 0; i < mine; ++i) {
      wait_lgkmcnt_0();  // the step before has been read
      asm volatile("" ::: "memory");
      if (i + 1 < mine) {
        load(i + 1);
        wait_vmcnt<FEW_LOADS>();
      } else {
        wait_vmcnt_0();
      }
      asm volatile("" ::: "memory");
      const uint8_t* const st = ring + (i & 1) * FEW_STEP;
      auto frag = [&](int at) {
        Frag f;
        f.h[0] = *reinterpret_cast<const i32x4*>(st + at + c0);
        f.h[1] = *reinterpret_cast<const i32x4*>(st + at + c1);
        return f;
      };
      const i32x4 wa = *reinterpret_cast<const i32x4*>(st + FEW_SA + words_at);
      const i32x4 wb = *reinterpret_cast<const i32x4*>(st + FEW_SB + words_at);
      const int scales_a[2] = {(int)__builtin_amdgcn_perm(wa[1], wa[0], pick), (int)__builtin_amdgcn_perm(wa[3], wa[2], pick)};
      const int scales_b[2] = {(int)__builtin_amdgcn_perm(wb[1], wb[0], pick), (int)__builtin_amdgcn_perm(wb[3], wb[2], pick)};
      Frag bf[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) bf[nt] = frag(Few::BM * ROW_BYTES + nt * 16 * ROW_BYTES);
      static_for<0, 4>([&](auto MT) {
        constexpr int mt = decltype(MT)::value;
        if (mt >= bands) return;
        const Frag af = frag(mt * 16 * ROW_BYTES);
        static_for<0, 8>([&](auto I) {
          constexpr int h = decltype(I)::value / 4, nt = decltype(I)::value % 4;
          acc[mt][nt] = mfma<mt, nt, h>(bf[nt], af, acc[mt][nt], scales_b[nt / 2], scales_a[mt / 2]);
        });
      });
    }
    // The waves' sums, a band a wave.
    auto sums_of = [&](int w) { return reinterpret_cast<f32x4*>(lds + w * 2 * FEW_STEP); };
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        if (mt < bands) sums_of(wave)[(mt * 4 + nt) * 64 + lane] = acc[mt][nt];
    __syncthreads();
    uint32_t valid;
    if constexpr (KIND == KIND_CONTIGUOUS)
      valid = (uint32_t)(__builtin_amdgcn_ballot_w64(id == cur.group) >> (16 * wave)) & 0xFFFFu;
    else
      valid = band_rows<Few, KIND>(cur, RowMask{0, 0}, 16 * wave, 0);
    if (wave < bands && valid != 0) {
      f32x4 v[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        v[nt] = sums_of(0)[(wave * 4 + nt) * 64 + lane];
#pragma unroll
        for (int w = 1; w < Few::NW; ++w) v[nt] += sums_of(w)[(wave * 4 + nt) * 64 + lane];
      }
      store_band(cur.d + (size_t)(cur.m0 + 16 * wave) * p.n + cur.n0, p.n, valid, v, lane);
    }
    __syncthreads();  // the sums have been read
  }
}

}  // namespace mx

// Tiles of 64 x 64 up to which a call takes those: three rounds of a whole chip's. In us,
// with these and with the large ones: 512 x 2048 x 7168 (256 tiles) 10.1, 42.5; 1024 x 1024
// x 1024 (256) 4.7, 12.9; 16 x 2176 x 2432 (34) 4.8, 14.0; 12 groups of 16 x 2304 x 640 (432)
// 5.8, 8.1; 18 of 8 x 2304 x 5632 (648) 22.4, 26.6; single rows of 8 groups among 128,
// without padding, x 2048 x 7168 (256) 14.4, 39.9, and of 40 among 128 (1280) 56.8, 77.9, x
// 2048 x 2048 23.7, 23.8; 2048^3 (1024) 15.6, 18.4; 8 of up to 256 x 2048 x 2048 (1024) 20.0, 18.8; 16 of up to 32 x 7168 x 2048 (1792) 28.1, 25.3; 2048 x
// 4096 x 4096 (2048) 44.8, 29.8. (Not by dg_get_num_cus(): the order of the sums differs.)
constexpr long long FEW_TILES = 768;

// Tiles that a call may have, of C's size.
template <class C>
static long long most_tiles(int kind, const GemmArgs& p) {
  const long long m_blocks = (p.m + C::BM - 1) / C::BM, n_blocks = (p.n + C::BN - 1) / C::BN;
  const long long held = std::min(p.num_groups, p.m);  // groups that can have rows
  switch (kind) {
    case KIND_MASKED:  // an upper bound for the grid's size, as for no padding; the kernel counts the tiles
      return p.num_groups * m_blocks * n_blocks;
    case KIND_NOPAD:  // a row block for each of them, and one for each BM of the other rows
      return (held + (p.m - held) / C::BM) * n_blocks;
    case KIND_CONTIGUOUS:
      return C::SLOTS * m_blocks * n_blocks;
    default:
      return m_blocks * n_blocks;
  }
}

template <int KIND>
static hipError_t launch_few(GemmArgs args, int num_cus, hipStream_t stream) {
  using C = mx::Few;
  args.m_blocks = (args.m + C::BM - 1) / C::BM;
  args.n_blocks = args.n / C::BN;
  args.num_tiles = (int)most_tiles<C>(KIND, args);
  const int grid = std::min(args.num_tiles, num_cus);
  hipLaunchKernelGGL(mx::fp4_gemm_few_kernel<KIND>, dim3(grid), dim3(C::THREADS), 0, stream, args);
  return hipGetLastError();
}

template <class C, int KIND>
static hipError_t launch_tiles(GemmArgs args, int num_cus, hipStream_t stream) {
  args.m_blocks = (args.m + C::BM - 1) / C::BM;
  args.n_blocks = (args.n + C::BN - 1) / C::BN;
  args.num_tiles = (int)most_tiles<C>(KIND, args);
  auto kern = mx::fp4_gemm_nt_kernel<C, KIND>;
  int per_cu = 1;
  hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kern, C::THREADS, 0);
  if (e != hipSuccess) return e;
  if (per_cu < 1) per_cu = 1;
  const int grid = balanced_grid(args.num_tiles, (long long)num_cus * per_cu);
  if (grid < 1) return hipSuccess;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(C::THREADS), 0, stream, args);
  return hipGetLastError();
}

// Tiles of 128 x 256 up to which a call takes those, one to a compute unit: 2048 x 4096 x
// 4096 (256) 23.9 us, with 256 x 256 30.0; 2048^3 (128) 13.9, 18.5; 8 groups of up to 256 x
// 2048 x 2048 (128) 14.5, 18.5; but 3000 x 4096 x 2048 (384) 25.0, 19.9. So do masked calls
// of at most 128 rows a group, half of whose larger tiles would be empty: 32 groups of up
// to 64 x 4096 x 7168 92, 96; 29 of up to 48 x 2688 x 640 12.6, 13.5; but 32 of up to 256 x
// 4096 x 7168 163, 131.
constexpr long long HALF_TILES = 256;

template <int KIND>
static hipError_t launch_mx(const GemmArgs& args, int num_cus, hipStream_t stream) {
  if (most_tiles<mx::Few>(KIND, args) <= FEW_TILES) return launch_few<KIND>(args, num_cus, stream);
  if (most_tiles<mx::Half>(KIND, args) <= HALF_TILES || (KIND == KIND_MASKED && args.m <= mx::Half::BM))
    return launch_tiles<mx::Half, KIND>(args, num_cus, stream);
  return launch_tiles<mx::Big, KIND>(args, num_cus, stream);
}

hipError_t launch_fp4(int kind, GemmArgs args, int num_cus, hipStream_t stream) {
  switch (kind) {
    case KIND_MASKED:
      return launch_mx<KIND_MASKED>(args, num_cus, stream);
    case KIND_NOPAD:
      return launch_mx<KIND_NOPAD>(args, num_cus, stream);
    case KIND_CONTIGUOUS:
      return launch_mx<KIND_CONTIGUOUS>(args, num_cus, stream);
    default:
      return launch_mx<KIND_DENSE>(args, num_cus, stream);
  }
}

}  // namespace dg
