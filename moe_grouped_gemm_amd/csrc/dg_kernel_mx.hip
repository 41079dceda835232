// FP4 NT GEMM with one E8M0 scale per 32 values of either operand (MXFP4) and
// BF16 output, dense and M-grouped, for gfx950 (MI355X):
//
//   D[m][n] = bf16( sum_k e2m1(A[m][k]) 2^(ea[m][k/32] - 127) * e2m1(B[n][k]) 2^(eb[n][k/32] - 127) )
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes packed E2M1 for both operands: lane
// group g = lane / 16 holds K positions 32g .. 32g + 31 of row lane % 16 (16
// bytes, even k in the low nibble), which are one scale block, and applies the
// block's two scales itself. Its float32 accumulator holds the sums: no step of
// the kernel's own follows the products but the one rounding to BF16.
//
// A persistent kernel over 256 x 256 tiles; a K step is 256 values, 128-byte rows of
// either operand, in one of two LDS stages that direct-to-LDS loads fill one to two
// steps ahead, with one barrier a step (see the K loop): the pipeline of
// dg_kernel.hip, whose stages hold as many bytes and half the values.

#include "dg_device.h"

namespace dg {
namespace mx {

struct Cfg {
  static constexpr int BM = 256, BN = 256, SLOTS = BM / 128;
  static constexpr int WAVES_N = 4, NW = 8, THREADS = NW * 64;
  static constexpr int WM = 128, WN = 64, MT = WM / 16, NT = WN / 16;
};
constexpr int STEP_BLOCKS = 2;                          // 128-value blocks of K a step: 128-byte rows
constexpr int A_BYTES = Cfg::BM * ROW_BYTES;            // 32 KB
constexpr int B_BYTES = Cfg::BN * ROW_BYTES;            // 32 KB
constexpr int SA_OFF = A_BYTES + B_BYTES;               // [block of the step][256] LHS scale words
constexpr int SB_OFF = SA_OFF + STEP_BLOCKS * Cfg::BM * 4;
constexpr int STAGE_BYTES = SB_OFF + STEP_BLOCKS * Cfg::BN * 4;
static_assert(Cfg::NW == 8 && Cfg::BM == 256 && Cfg::BN == 256, "load split below");

}  // namespace mx

template <>
constexpr int A_PACK_SHIFT<mx::Cfg> = 1;

namespace mx {

// One LDS buffer per stage, and its byte address.
template <int S>
__device__ __forceinline__ uint8_t* stage_buf() {
  __shared__ __attribute__((aligned(1024))) uint8_t buf[STAGE_BYTES];
  return buf;
}
template <int S>
__device__ __forceinline__ uint32_t stage_addr() {
  return (uint32_t)(uintptr_t)(lds_void*)stage_buf<S>();
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 4, voff, 0, 0, 0);
}

// This lane's byte offsets within a tile: of its A and B loads (the j-th adds 64 j
// rows) and of its scale words.
struct LaneOffsets {
  uint32_t ab, ab_step, sc;
};

__device__ __forceinline__ LaneOffsets lane_offsets(int k, int wave, int lane) {
  LaneOffsets o;
  const int row0 = wave * 8 + (lane >> 3);
  o.ab = (uint32_t)row0 * ((uint32_t)k / 2) + (uint32_t)(((lane & 7) ^ ((row0 >> 1) & 7)) * 16);  // the same for every j
  o.ab_step = 64u * ((uint32_t)k / 2);
  o.sc = (uint32_t)(64 * (wave & 3) + lane) * 4u;
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

__device__ __forceinline__ TileSrc tile_src(const GemmArgs& p, const TileRef& tr) {
  TileSrc s;
  const size_t row = (size_t)p.k / 2;
  s.a_rows = uniform_int(min(max(tr.load_rows - tr.m0, 0), Cfg::BM));
  s.b_rows = uniform_int(min(p.n - tr.n0, Cfg::BN));
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
struct StageSrc {
  __amdgpu_buffer_rsrc_t a, b, sa, sb;
};

__device__ __forceinline__ StageSrc stage_src(const GemmArgs& p, const TileSrc& t, int step, int wave) {
  StageSrc r;
  const uint32_t row = (uint32_t)p.k / 2, skip = (uint32_t)step * ROW_BYTES;
  const int blk = step * STEP_BLOCKS + (wave >> 2);  // the 128-value block whose scales this wave loads
  const bool in = blk < p.k / BK;
  r.a = buffer_rsrc(t.a + skip, t.a_rows ? t.a_rows * row - skip : 0);
  r.b = buffer_rsrc(t.b + skip, t.b_rows * row - skip);
  r.sa = buffer_rsrc(t.sa + (size_t)blk * p.ld_sfa, in ? t.a_rows * 4u : 0);
  r.sb = buffer_rsrc(t.sb + (size_t)blk * p.ld_sfb, in ? t.b_rows * 4u : 0);
  return r;
}

// Descriptors of the step `ahead` steps after step 0 of the current tile: a step of
// this tile, of the next one, or (with a single step per tile) of the one after.
// With no such tile the window's entries repeat the previous one and the loads fetch
// a step nobody reads.
__device__ __forceinline__ StageSrc refill_src(const GemmArgs& p, const TileSrc& t0, const TileSrc& t1,
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
  return stage_src(p, t, in0 ? ahead : (in1 ? ahead - steps : ahead - 2 * steps), wave);
}

// The loads of one step into stage S, in four parts (see the K loop): 0 and 1 the A
// tile, 2 and 3 the B tile, 3 also the scale words.
template <int S, int PART>
__device__ __forceinline__ void issue_part(const StageSrc& r, int wave, const LaneOffsets& lo) {
  const uint32_t st = stage_addr<S>();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = PART % 2 * 2 + i;
    dma16(PART < 2 ? r.a : r.b, lo.ab + j * lo.ab_step, st + (PART < 2 ? 0 : A_BYTES) + (j * Cfg::NW + wave) * 1024);
  }
  if constexpr (PART == 3) {
    const int at = ((wave >> 2) * 256 + 64 * (wave & 3)) * 4;
    dma4(r.sa, lo.sc, st + SA_OFF + at);
    dma4(r.sb, lo.sc, st + SB_OFF + at);
  }
}

// A lane's LDS byte offsets within a stage, fixed for the kernel (a 16-row band adds
// 2048 bytes; see lds_offset() for the swizzle).
struct LdsOffsets {
  uint32_t a0, a1, b0, b1;  // the pieces of K block 0 and 1 of the step, of the wave's first band or columns
  uint32_t sa, sb;          // its words, 64 rows a read
};

__device__ __forceinline__ LdsOffsets lds_offsets(int wm0, int wn0, int lane) {
  LdsOffsets o;
  const int r = lane & 15, g = lane >> 4;
  const uint32_t c0 = (uint32_t)lds_offset(r, g), c1 = (uint32_t)lds_offset(r, g + 4);
  o.a0 = (uint32_t)wm0 * ROW_BYTES + c0;
  o.a1 = (uint32_t)wm0 * ROW_BYTES + c1;
  o.b0 = A_BYTES + (uint32_t)wn0 * ROW_BYTES + c0;
  o.b1 = A_BYTES + (uint32_t)wn0 * ROW_BYTES + c1;
  o.sa = SA_OFF + (uint32_t)(wm0 + lane) * 4;
  o.sb = SB_OFF + (uint32_t)(wn0 + lane) * 4;
  return o;
}

// A 16-row fragment of both K blocks of a step: piece g of the row's first half and of
// its second.
struct Frag {
  i32x4 h[STEP_BLOCKS];
};
template <int S>
__device__ __forceinline__ Frag frag_at(uint32_t off0, uint32_t off1, int band) {
  const uint8_t* st = stage_buf<S>();
  Frag f;
  f.h[0] = *reinterpret_cast<const i32x4*>(st + off0 + band * 16 * ROW_BYTES);
  f.h[1] = *reinterpret_cast<const i32x4*>(st + off1 + band * 16 * ROW_BYTES);
  return f;
}
__device__ __forceinline__ i32x8 operand(const i32x4& v) { return (i32x8){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The scale words of a wave's rows and columns as they lie in LDS, lane l the word of
// the l-th of 64 rows: of either K block, rows 0 .. 63 and 64 .. 127, and the columns.
struct Words {
  uint32_t a[STEP_BLOCKS][2], b[STEP_BLOCKS];
};
template <int S>
__device__ __forceinline__ Words words_at(const LdsOffsets& lds) {
  const uint8_t* st = stage_buf<S>();
  Words w;
#pragma unroll
  for (int h = 0; h < STEP_BLOCKS; ++h) {
    w.a[h][0] = *reinterpret_cast<const uint32_t*>(st + lds.sa + h * 1024);
    w.a[h][1] = *reinterpret_cast<const uint32_t*>(st + lds.sa + h * 1024 + 256);
    w.b[h] = *reinterpret_cast<const uint32_t*>(st + lds.sb + h * 1024);
  }
  return w;
}

// Lane (r, g) of four groups of 16 gives the scale word of row 16g + r, and gets
// byte g of the words of rows r, 16 + r, 32 + r and 48 + r: the codes of its K
// positions in four successive 16-row fragments, in the order in which the
// MFMA's byte select counts.
__device__ __forceinline__ int scale_codes(uint32_t w, uint32_t pick_lo, uint32_t pick_hi) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 half = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const u32x2 lo = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
  const u32x2 hi = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
  return (int)(__builtin_amdgcn_perm(lo[1], lo[0], pick_lo) | __builtin_amdgcn_perm(hi[1], hi[0], pick_hi));
}
struct Codes {
  int a[STEP_BLOCKS][2], b[STEP_BLOCKS];
};
__device__ __forceinline__ Codes codes_of(const Words& w, int lane) {
  const uint32_t g = lane >> 4;
  const uint32_t pick_lo = g | (4 + g) << 8 | 0x0C0C0000u, pick_hi = 0x0C0Cu | g << 16 | (4 + g) << 24;
  Codes c;
#pragma unroll
  for (int h = 0; h < STEP_BLOCKS; ++h) {
    c.a[h][0] = scale_codes(w.a[h][0], pick_lo, pick_hi);
    c.a[h][1] = scale_codes(w.a[h][1], pick_lo, pick_hi);
    c.b[h] = scale_codes(w.b[h], pick_lo, pick_hi);
  }
  return c;
}

template <int MT, int NT, int H>
__device__ __forceinline__ f32x4 mfma(const Frag& b, const Frag& a, const f32x4& c, const Codes& s) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.h[H]), operand(a.h[H]), c, 4, 4, NT, s.b[H], MT & 3,
                                                          s.a[H][MT >> 2]);
}

// Writes a wave's finished 128 x 64 sub-tile as BF16 (round to nearest even), valid rows
// only. Each 16-row band goes through LDS, so that every store covers whole 128-byte
// row segments (8 lanes per row), in two of this wave's own 1 KB B slots of stage S,
// the stage the tile's last step read: no wave reads it again before the next barrier,
// and only this wave's own refill loads, issued later, overwrite these slots. 16-byte
// slots are XOR-swizzled by row.
template <int KIND, int S>
__device__ __forceinline__ void store_tile(const GemmArgs& p, const TileRef& cur, const RowMask& cm,
                                           const f32x4 (&acc)[Cfg::MT][Cfg::NT], int wave, int wm0, int wn0,
                                           int lane) {
  static_assert(Cfg::WN * 2 == ROW_BYTES, "one 128-byte row segment per wave and row");
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  uint8_t* const st = stage_buf<S>();
  const int wbase = A_BYTES + wave * 1024;  // slot j of the wave at + j * NW * 1024
  const int r = lane & 15, q = lane >> 4;
  auto slot_off = [](int row, int sl) { return (row >> 3) * Cfg::NW * 1024 + (row & 7) * 128 + ((sl ^ (row & 7)) << 4); };
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) {
    const uint32_t valid = band_rows<Cfg, KIND>(cur, cm, wm0, mt);
    if (valid == 0) continue;
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt) {
      const f32x4 v = acc[mt][nt];
      const i32x2 packed = {(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
      // columns 16 nt + 4 q .. + 3: half (q & 1) of 16-byte slot 2 nt + q / 2
      *reinterpret_cast<i32x2*>(st + (wbase + slot_off(r, 2 * nt + (q >> 1)) + (q & 1) * 8)) = packed;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = (lane >> 3) + 8 * half;
      const int sl = lane & 7;
      const i32x4 v = *reinterpret_cast<const i32x4*>(st + (wbase + slot_off(row, sl)));
      if ((valid >> row) & 1) {
        uint16_t* drow = cur.d + (size_t)(cur.m0 + wm0 + mt * 16 + row) * p.n + cur.n0 + wn0 + 8 * sl;
        if constexpr (KIND == KIND_DENSE) *(global_i32x4*)drow = v;
        else __builtin_nontemporal_store(v, (global_i32x4*)drow);
      }
    }
  }
}

// The K loop of one tile; its first step reads stage PHASE. Step i of the global
// sequence of steps reads stage s = i % 2:
//   entry:     the first step's operands are read (its stage was completed before the
//              last barrier);
//   bands 0-5: the A fragment two bands ahead from stage s, 8 MFMAs of the band (4
//              column blocks, 2 K blocks); bands 0 and 1 also issue parts 2 and 3 of the
//              refill of stage 1 - s (step i + 1);
//   barrier:   after it every wave's loads of step i + 1 have landed and no wave reads
//              stage s any more (bands 6 and 7 work from registers);
//   bands 6-7: column block by column block, so that a B fragment is read again for step
//              i + 1 as soon as its last MFMA of step i has issued, then the next step's
//              first A fragments and its scale words; parts 0 and 1 of the refill of stage
//              s (step i + 2) are issued.
// Only bands below NB are computed (the rows of the others are not stored).
template <int KIND, int PHASE, int NB>
__device__ __forceinline__ void mainloop(const GemmArgs& p, const TileSrc& t0, const TileSrc& t1, const TileSrc& t2,
                                         f32x4 (&acc)[Cfg::MT][Cfg::NT], bool on, int wave, int lane,
                                         const LdsOffsets& lds, const LaneOffsets& lo, const RowGroups& nrg, int ngroup,
                                         RowMask& nmask) {
  static_assert(NB == Cfg::MT || (NB >= 2 && NB <= 6), "a partial copy computes bands 0 .. NB-1 before the barrier");
  // The next tile's row mask (contiguous layout), after a barrier: see RowGroups.
  auto next_rows = [&]() {
    if constexpr (KIND == KIND_CONTIGUOUS) {
      int e = nrg.even, o = nrg.odd;
      asm volatile("" : "+v"(e), "+v"(o));  // keeps the compare (and the wait for the loads) here
      nmask = row_mask(RowGroups{e, o}, ngroup);
    }
  };
  const int steps = (p.k / BK + STEP_BLOCKS - 1) / STEP_BLOCKS;
  Frag af[4], bf[Cfg::NT];  // A ring: band mt's fragment in slot mt % 4
#pragma unroll
  for (int nt = 0; nt < Cfg::NT; ++nt) bf[nt] = frag_at<PHASE>(lds.b0, lds.b1, nt);
  af[0] = frag_at<PHASE>(lds.a0, lds.a1, 0);
  af[1] = frag_at<PHASE>(lds.a0, lds.a1, 1);
  Words words = words_at<PHASE>(lds);
  for (int i0 = 0; i0 < steps; i0 += 2) {
    static_for<0, 2>([&](auto si) {
      constexpr int s = (decltype(si)::value + PHASE) % 2, sn = 1 - s;
      const int i = i0 + decltype(si)::value;
      if (i >= steps) return;
      // The refills are issued unconditionally (past the last tile they load a step nobody
      // reads): a branch here would make the compiler wait for them before reading the
      // current stage.
      const StageSrc r1 = refill_src(p, t0, t1, t2, i + 1, steps, wave);
      const StageSrc r2 = refill_src(p, t0, t1, t2, i + 2, steps, wave);
      if (!on) {
        issue_part<sn, 2>(r1, wave, lo);
        issue_part<sn, 3>(r1, wave, lo);
        wait_vmcnt_0();
        wait_lgkmcnt_0();
        barrier();
        next_rows();
        issue_part<s, 0>(r2, wave, lo);
        issue_part<s, 1>(r2, wave, lo);
        return;
      }
      const Codes codes = codes_of(words, lane);
      static_for<0, 6>([&](auto MT) {
        constexpr int mt = decltype(MT)::value;
        if constexpr (mt + 2 < NB) af[(mt + 2) % 4] = frag_at<s>(lds.a0, lds.a1, mt + 2);
        if constexpr (mt == 0) issue_part<sn, 2>(r1, wave, lo);
        if constexpr (mt == 1) issue_part<sn, 3>(r1, wave, lo);
        if constexpr (mt < NB) {
          static_for<0, STEP_BLOCKS * Cfg::NT>([&](auto I) {
            constexpr int h = decltype(I)::value / Cfg::NT, nt = decltype(I)::value % Cfg::NT;
            acc[mt][nt] = mfma<mt, nt, h>(bf[nt], af[mt % 4], acc[mt][nt], codes);
          });
          // The reads two bands ahead and this band's share of the refill first.
          if constexpr (mt + 2 < NB) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // DS reads
          if constexpr (mt == 0) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);      // VMEM loads
          if constexpr (mt == 1) __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, STEP_BLOCKS * Cfg::NT, 0);  // MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<0, Cfg::NT>([&](auto NT) {
        constexpr int nt = decltype(NT)::value;
        if constexpr (NB == Cfg::MT) {
          acc[6][nt] = mfma<6, nt, 0>(bf[nt], af[2], acc[6][nt], codes);
          acc[7][nt] = mfma<7, nt, 0>(bf[nt], af[3], acc[7][nt], codes);
          acc[6][nt] = mfma<6, nt, 1>(bf[nt], af[2], acc[6][nt], codes);
          acc[7][nt] = mfma<7, nt, 1>(bf[nt], af[3], acc[7][nt], codes);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (nt == 0) {
          wait_lgkmcnt_0();
          wait_vmcnt_0();
          barrier();
          next_rows();
          __builtin_amdgcn_sched_barrier(0);
          issue_part<s, 0>(r2, wave, lo);
        }
        if constexpr (nt == 1) issue_part<s, 1>(r2, wave, lo);
        // The next step's operands (past a tile's last step: the next tile's first, which
        // its entry reads again).
        bf[nt] = frag_at<sn>(lds.b0, lds.b1, nt);
        if constexpr (nt == 1) af[0] = frag_at<sn>(lds.a0, lds.a1, 0);
        if constexpr (nt == 2) words = words_at<sn>(lds);
        if constexpr (nt == 3) af[1] = frag_at<sn>(lds.a0, lds.a1, 1);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }
}

// A wave whose valid rows lie in its first HALF_BANDS bands runs a copy of the K loop
// without the other bands' MFMAs (their rows are never stored).
constexpr int HALF_BANDS = 4;

template <int KIND>
__global__ void __launch_bounds__(Cfg::THREADS, 1) fp4_gemm_nt_kernel(GemmArgs p) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / Cfg::WAVES_N) * Cfg::WM;
  const int wn0 = (wave % Cfg::WAVES_N) * Cfg::WN;
  const int steps = (p.k / BK + STEP_BLOCKS - 1) / STEP_BLOCKS;

  int num_tiles = p.num_tiles;
  [[maybe_unused]] int* s_prefix = nullptr;
  if constexpr (counts_on_device(KIND)) {
    s_prefix = group_table<Cfg, KIND>(p, tid);
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
  TileRef cur = next_active<Cfg, KIND>(p, t, grid, num_tiles, s_prefix);
  if (!cur.active) return;
  int t1 = t + grid;
  TileRef nxt = next_active<Cfg, KIND>(p, t1, grid, num_tiles, s_prefix);
  int t2 = t1 + grid;
  TileRef nx2;
  nx2.active = false;
  if (nxt.active) nx2 = next_active<Cfg, KIND>(p, t2, grid, num_tiles, s_prefix);
  const LaneOffsets lo = lane_offsets(p.k, wave, lane);
  const LdsOffsets lds = lds_offsets(wm0, wn0, lane);
  TileSrc c0 = tile_src(p, cur);
  TileSrc c1 = nxt.active ? tile_src(p, nxt) : c0;
  TileSrc c2 = nx2.active ? tile_src(p, nx2) : c1;

  // The first tile's row groups (contiguous layout) are loaded before the prologue's
  // loads, so that waiting for them never waits for those.
  [[maybe_unused]] RowGroups crg{-1, -1};
  if constexpr (KIND == KIND_CONTIGUOUS) crg = load_row_groups<Cfg>(p, cur, wm0, lane);

  // Step 0 into stage 0 and parts 0 and 1 of step 1 into stage 1 (the first step issues
  // the rest); step 0 must have landed for every wave before it is read.
  {
    const StageSrc r0 = refill_src(p, c0, c1, c2, 0, steps, wave);
    const StageSrc r1 = refill_src(p, c0, c1, c2, 1, steps, wave);
    issue_part<0, 0>(r0, wave, lo);
    issue_part<0, 1>(r0, wave, lo);
    issue_part<0, 2>(r0, wave, lo);
    issue_part<0, 3>(r0, wave, lo);
    issue_part<1, 0>(r1, wave, lo);
    issue_part<1, 1>(r1, wave, lo);
    wait_vmcnt<4>();  // all but step 1's parts 0 and 1
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
    int bands = Cfg::MT;
    if constexpr (counts_on_device(KIND))
      bands = uniform_int(min(max((cur.valid_rows - cur.m0 - wm0 + 15) / 16, 0), Cfg::MT));
    RowGroups nrg{-1, -1};
    if constexpr (KIND == KIND_CONTIGUOUS) nrg = load_row_groups<Cfg>(p, nxt, wm0, lane);
    f32x4 acc[Cfg::MT][Cfg::NT];
#pragma unroll
    for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < Cfg::NT; ++nt) acc[mt][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};

    if (counts_on_device(KIND) && bands <= HALF_BANDS) {
      if (phase == 0) mainloop<KIND, 0, HALF_BANDS>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
      else mainloop<KIND, 1, HALF_BANDS>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
    } else {
      if (phase == 0) mainloop<KIND, 0, Cfg::MT>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
      else mainloop<KIND, 1, Cfg::MT>(p, c0, c1, c2, acc, on, wave, lane, lds, lo, nrg, nxt.group, nmask);
    }
    phase = (phase + steps) & 1;

    // Epilogue (the next tile's first step has landed, its second is in flight), from the
    // stage the tile's last step read.
    if (on) {
      if (phase == 0) store_tile<KIND, 1>(p, cur, cmask, acc, wave, wm0, wn0, lane);
      else store_tile<KIND, 0>(p, cur, cmask, acc, wave, wm0, wn0, lane);
    }
    // Slide the window.
    cmask = nmask;
    cur = nxt;
    c0 = c1;
    nxt = nx2;
    c1 = c2;
    if (nx2.active) {
      t2 += grid;
      nx2 = next_active<Cfg, KIND>(p, t2, grid, num_tiles, s_prefix);
    }
    c2 = nx2.active ? tile_src(p, nx2) : c1;
  }
  // The last refills loaded steps nobody reads; no wave may end while such a load can
  // still write its LDS.
  wait_vmcnt_0();
}

}  // namespace mx

template <int KIND>
static hipError_t launch_mx(const GemmArgs& args, int num_cus, hipStream_t stream) {
  auto kern = mx::fp4_gemm_nt_kernel<KIND>;
  int per_cu = 1;
  hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kern, mx::Cfg::THREADS, 0);
  if (e != hipSuccess) return e;
  if (per_cu < 1) per_cu = 1;
  const int grid = balanced_grid(args.num_tiles, (long long)num_cus * per_cu);
  if (grid < 1) return hipSuccess;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(mx::Cfg::THREADS), 0, stream, args);
  return hipGetLastError();
}

hipError_t launch_fp4(int kind, GemmArgs args, int num_cus, hipStream_t stream) {
  using C = mx::Cfg;
  args.m_blocks = (args.m + C::BM - 1) / C::BM;
  args.n_blocks = (args.n + C::BN - 1) / C::BN;
  switch (kind) {
    case KIND_MASKED:  // an upper bound for the grid's size, as for no padding; the kernel counts the tiles
      args.num_tiles = args.num_groups * args.m_blocks * args.n_blocks;
      return launch_mx<KIND_MASKED>(args, num_cus, stream);
    case KIND_NOPAD:  // each group adds at most one partial row block
      args.num_tiles = (args.m_blocks + args.num_groups) * args.n_blocks;
      return launch_mx<KIND_NOPAD>(args, num_cus, stream);
    case KIND_CONTIGUOUS:
      args.num_tiles = C::SLOTS * args.m_blocks * args.n_blocks;
      return launch_mx<KIND_CONTIGUOUS>(args, num_cus, stream);
    default:
      args.num_tiles = args.m_blocks * args.n_blocks;
      return launch_mx<KIND_DENSE>(args, num_cus, stream);
  }
}

}  // namespace dg
