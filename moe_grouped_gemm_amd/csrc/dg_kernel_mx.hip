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
// Per 256 x 256 tile a double-buffered loop over 256 values of K loads A and B
// (128-byte rows) and the scale words straight into LDS.

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

__device__ __forceinline__ uint8_t* lds() {
  __shared__ __attribute__((aligned(1024))) uint8_t buf[2 * STAGE_BYTES];
  return buf;
}
__device__ __forceinline__ uint32_t lds_addr() { return (uint32_t)(uintptr_t)(lds_void*)lds(); }

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds_dest(lds_base), 4, voff, 0, 0, 0);
}

// Where a tile's operands start (the group's B and its scales are located from
// the group index).
struct Src {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  uint32_t a_rows, b_rows;
};

template <int KIND>
__device__ __forceinline__ Src tile_src(const GemmArgs& p, const TileRef& tr) {
  Src s;
  const size_t row = (size_t)p.k / 2;
  s.a_rows = (uint32_t)min(max(tr.load_rows - tr.m0, 0), Cfg::BM);
  s.b_rows = (uint32_t)min(p.n - tr.n0, Cfg::BN);
  s.a = tr.a + (size_t)tr.m0 * row;
  s.sa = tr.sfa + tr.m0;
  s.b = p.b + ((size_t)tr.group * p.n + tr.n0) * row;
  s.sb = p.sfb + (size_t)tr.group * (p.k / BK) * p.ld_sfb + tr.n0;
  return s;
}

// Loads of the 256 values from block kb on into the stage at LDS byte address
// st. Wave w: A and B rows w * 8 + lane / 8 + 64 j (j < 4, 16 bytes each, with
// the swizzle of lds_offset()); scale words: block w / 4 of the step, rows 64
// (w % 4) + lane. Rows past the matrix read as zero. So does everything of an odd
// last block's second half: the scale words by their descriptors, and codes
// that are rows' first values or other rows' (no code is infinite or NaN) come
// to nothing under two scales of 2^-127.
__device__ __forceinline__ void issue_step(const GemmArgs& p, const Src& s, int kb, uint32_t st, int wave, int lane,
                                           uint32_t lane_off) {
  const uint32_t row = (uint32_t)p.k / 2, skip = (uint32_t)kb * (BK / 2);
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(s.a + skip, s.a_rows ? s.a_rows * row - skip : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) dma16(ra, lane_off + (uint32_t)j * 64u * row, st + (j * Cfg::NW + wave) * 1024);
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(s.b + skip, s.b_rows * row - skip);
#pragma unroll
  for (int j = 0; j < 4; ++j) dma16(rb, lane_off + (uint32_t)j * 64u * row, st + A_BYTES + (j * Cfg::NW + wave) * 1024);
  const int blk = wave >> 2, q = wave & 3;
  const bool in = kb + blk < p.k / BK;
  const uint32_t at = (uint32_t)(64 * q + lane) * 4u;
  const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(s.sa + (size_t)(kb + blk) * p.ld_sfa, in ? s.a_rows * 4u : 0);
  dma4(rsa, at, st + SA_OFF + (blk * Cfg::BM + 64 * q) * 4);
  const __amdgpu_buffer_rsrc_t rsb = buffer_rsrc(s.sb + (size_t)(kb + blk) * p.ld_sfb, in ? s.b_rows * 4u : 0);
  dma4(rsb, at, st + SB_OFF + (blk * Cfg::BN + 64 * q) * 4);
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

__device__ __forceinline__ i32x8 operand(i32x4 v) { return (i32x8){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// One step of a wave's 128 x 64 sub-tile from the stage at `st`, bands 0 ..
// NB-1 (the rows of the others are not stored).
template <int NB>
__device__ __forceinline__ void step(f32x4 (&acc)[Cfg::MT][Cfg::NT], const uint8_t* st, int wm0, int wn0, int lane) {
  const int r = lane & 15, g = lane >> 4;
  const uint32_t pick_lo = (uint32_t)g | (uint32_t)(4 + g) << 8 | 0x0C0C0000u;
  const uint32_t pick_hi = 0x0C0Cu | (uint32_t)g << 16 | (uint32_t)(4 + g) << 24;
  static_for<0, STEP_BLOCKS>([&](auto H) {
    constexpr int h = decltype(H)::value;
    auto words = [&](int off, int row) {
      return *reinterpret_cast<const uint32_t*>(st + off + (h * 256 + row + lane) * 4);
    };
    int ea[2];
    ea[0] = scale_codes(words(SA_OFF, wm0), pick_lo, pick_hi);
    ea[1] = scale_codes(words(SA_OFF, wm0 + 64), pick_lo, pick_hi);
    const int eb = scale_codes(words(SB_OFF, wn0), pick_lo, pick_hi);
    i32x8 bf[Cfg::NT];
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt)
      bf[nt] = operand(*reinterpret_cast<const i32x4*>(st + A_BYTES + lds_offset(wn0 + nt * 16 + r, 4 * h + g)));
    auto read_a = [&](int mt) {
      return operand(*reinterpret_cast<const i32x4*>(st + lds_offset(wm0 + mt * 16 + r, 4 * h + g)));
    };
    i32x8 af[2];
    af[0] = read_a(0);
    static_for<0, NB>([&](auto MT) {
      constexpr int mt = decltype(MT)::value;
      if constexpr (mt + 1 < NB) af[(mt + 1) & 1] = read_a(mt + 1);
      static_for<0, Cfg::NT>([&](auto NT) {
        constexpr int nt = decltype(NT)::value;
        acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[nt], af[mt & 1], acc[mt][nt], 4, 4, nt, eb,
                                                                       mt & 3, ea[mt >> 2]);
      });
    });
  });
}

// Writes a wave's finished 128 x 64 sub-tile as BF16 (round to nearest even),
// valid rows only, each 16-row band through 2 KB of LDS of the wave's own (`scr`) so
// that every store covers a whole 128-byte row segment (8 lanes per row); 16-byte
// slots are XOR-swizzled by row.
template <int KIND>
__device__ __forceinline__ void store_tile(const GemmArgs& p, const TileRef& cur, const RowMask& cm,
                                           const f32x4 (&acc)[Cfg::MT][Cfg::NT], uint8_t* scr, int wm0, int wn0,
                                           int lane) {
  static_assert(Cfg::WN * 2 == ROW_BYTES, "one 128-byte row segment per wave and row");
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const int r = lane & 15, q = lane >> 4;
  auto slot_off = [](int row, int sl) { return row * ROW_BYTES + ((sl ^ (row & 7)) << 4); };
#pragma unroll
  for (int mt = 0; mt < Cfg::MT; ++mt) {
    const uint32_t valid = band_rows<Cfg, KIND>(cur, cm, wm0, mt);
    if (valid == 0) continue;
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt) {
      const f32x4 v = acc[mt][nt];
      const i32x2 packed = {(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
      // columns 16 nt + 4 q .. + 3: half (q & 1) of 16-byte slot 2 nt + q / 2
      *reinterpret_cast<i32x2*>(scr + slot_off(r, 2 * nt + (q >> 1)) + (q & 1) * 8) = packed;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = (lane >> 3) + 8 * half;
      const int sl = lane & 7;
      const i32x4 v = *reinterpret_cast<const i32x4*>(scr + slot_off(row, sl));
      if ((valid >> row) & 1) {
        uint16_t* drow = cur.d + (size_t)(cur.m0 + wm0 + mt * 16 + row) * p.n + cur.n0 + wn0 + 8 * sl;
        if constexpr (KIND == KIND_DENSE) *(global_i32x4*)drow = v;
        else __builtin_nontemporal_store(v, (global_i32x4*)drow);
      }
    }
  }
}

// Step i has landed for every wave after the wait and barrier at its top, and
// nobody reads the other stage any more. The wait is explicit: the compiler does
// not see the direct-to-LDS loads. The last step of a tile loads the first of the
// next.
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

  const int row0 = wave * 8 + (lane >> 3);
  const uint32_t lane_off =
      (uint32_t)row0 * ((uint32_t)p.k / 2) + (uint32_t)(((lane & 7) ^ ((row0 >> 1) & 7)) * 16);  // the same for every j

  const int grid = gridDim.x;
  int rank = blockIdx.x;
  if ((grid & 7) == 0) rank = (blockIdx.x & 7) * (grid >> 3) + (blockIdx.x >> 3);

  const uint32_t base = lds_addr();
  uint8_t* const buf = lds();
  int t = rank;
  TileRef cur = next_active<Cfg, KIND>(p, t, grid, num_tiles, s_prefix);
  if (!cur.active) return;
  Src src = tile_src<KIND>(p, cur);
  int stage = 0;  // the stage holding the current tile's first step
  issue_step(p, src, 0, base, wave, lane, lane_off);
  while (cur.active) {
    int tn = t + grid;
    const TileRef nxt = next_active<Cfg, KIND>(p, tn, grid, num_tiles, s_prefix);
    const Src nsrc = nxt.active ? tile_src<KIND>(p, nxt) : src;
    RowMask cm{0, 0};
    if constexpr (KIND == KIND_CONTIGUOUS) cm = row_mask(load_row_groups<Cfg>(p, cur, wm0, lane), cur.group);
    bool any_row;
    if constexpr (KIND == KIND_CONTIGUOUS) any_row = (cm.even | cm.odd) != 0;
    else any_row = cur.valid_rows > cur.m0 + wm0;
    const bool on = any_row && cur.n0 + wn0 < p.n;

    f32x4 acc[Cfg::MT][Cfg::NT];
#pragma unroll
    for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < Cfg::NT; ++nt) acc[mt][nt] = (f32x4){0.f, 0.f, 0.f, 0.f};

    for (int i = 0; i < steps; ++i) {
      const int cs = (stage + i) & 1;
      wait_vmcnt_0();
      __syncthreads();
      if (i + 1 < steps) issue_step(p, src, (i + 1) * STEP_BLOCKS, base + (cs ^ 1) * STAGE_BYTES, wave, lane, lane_off);
      else if (nxt.active) issue_step(p, nsrc, 0, base + (cs ^ 1) * STAGE_BYTES, wave, lane, lane_off);
      if (on) step<Cfg::MT>(acc, buf + cs * STAGE_BYTES, wm0, wn0, lane);
    }
    stage = (stage + steps) & 1;

    // The stage that the last step read is free once all have read it; it is loaded
    // again after the next step's barrier.
    __syncthreads();
    if (on) store_tile<KIND>(p, cur, cm, acc, buf + (stage ^ 1) * STAGE_BYTES + wave * 16 * ROW_BYTES, wm0, wn0, lane);
    cur = nxt;
    src = nsrc;
    t = tn;
  }
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
