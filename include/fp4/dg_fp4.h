/*
 * dg_fp4.h - products of FP4 (OCP E2M1) values with one power-of-two scale per
 * 32 of them, the microscaling format MXFP4, and its quantiser, for AMD
 * Instinct MI355X (gfx950). Same library (libdg.so), status codes, checks,
 * limits and conventions as dg.h: caller-owned device memory, nothing
 * allocated, arguments checked before anything is enqueued, one kernel a call on
 * `stream` of the current device, safe to capture in a HIP graph.
 */
#ifndef DG_FP4_H
#define DG_FP4_H

#include "../dg.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The products, dense and M-grouped. As the FP8 calls of the same layout in
 * dg.h, except for the operands and their scales:
 *   a   [m][k/2] bytes (masked [num_groups][max_m][k/2]) and
 *   b   [n][k/2] (grouped [num_groups][n][k/2]): E2M1 values packed two per
 *       byte along K, element 2j in the low nibble of byte j, as in the FP8 x
 *       FP4 calls
 *   sfa [k/128][dg_get_tma_aligned_size(m, 4)] words (masked: with the leading
 *       num_groups and max_m for m) and
 *   sfb [k/128][dg_get_tma_aligned_size(n, 4)] (grouped: with the leading
 *       num_groups): the four E8M0 codes of a row's 128 values, the code of
 *       the first 32 in the lowest byte; code e stands for 2^(e - 127), 255
 *       for NaN
 *   D = bf16( sum_k e2m1(A[m][k]) sfa[m][k/32] * e2m1(B[n][k]) sfb[n][k/32] )
 * Products accumulate in float32 inside the MFMA. dg_quantize_fp4 makes such
 * operands, dg_moe.h's steps the left ones of a mixture-of-experts block.
 * Fewer than 2^30 rows (masked: num_groups * max_m); a, b and d below 2^40 bytes each.
 */
dg_status dg_fp4_gemm_nt(const void* a, const uint32_t* sfa,
                         const void* b, const uint32_t* sfb,
                         void* d, int m, int n, int k, void* stream);
dg_status dg_m_grouped_fp4_gemm_nt_contiguous(const void* a, const uint32_t* sfa,
                                              const void* b, const uint32_t* sfb,
                                              void* d, const int32_t* grouped_layout,
                                              int m, int n, int k, int num_groups,
                                              void* stream);
dg_status dg_m_grouped_fp4_gemm_nt_masked(const void* a, const uint32_t* sfa,
                                          const void* b, const uint32_t* sfb,
                                          void* d, const int32_t* masked_m,
                                          int num_groups, int max_m, int n, int k,
                                          void* stream);
dg_status dg_m_grouped_fp4_gemm_nt_nopad(const void* a, const uint32_t* sfa,
                                         const void* b, const uint32_t* sfb,
                                         void* d, const int32_t* group_rows,
                                         int m, int n, int k, int num_groups,
                                         void* stream);

/* Element types of dg_quantize_fp4's input. */
#define DG_BF16 0
#define DG_FLOAT32 1

/*
 * Rows quantised to an operand of the FP4 GEMMs, and read back.
 *   x  [groups][rows][k] BF16 or, by x_type, float32 (read back: BF16)
 *   q  [groups][rows][k/2] bytes, sf [groups][k/128][dg_get_tma_aligned_size(rows, 4)]
 *      words, both as the GEMMs take them (groups = 1: one operand)
 * Per 32 values the scale is the smallest power of two that is not below
 * amax / 6, so that nothing saturates, and at least 2^-127; codes are
 * e2m1(x / scale), rounded to nearest, ties to the even code. (The conversion that the
 * microscaling text itself gives takes 2^(floor(log2 amax) - 2): half this scale where
 * amax is above 1.5 times its power of two, values above 6 times that cut to it. Its codes
 * differ there; the products take either.) An infinity or a NaN
 * makes its block's scale NaN, and with it all of its 32 values. Words past
 * the last row are not written. Read back, a value is exact, but for one past
 * BF16's largest, which becomes infinite (a value from 1.75 2^127 on rounds up to
 * 2^128).
 * rows and groups may be 0; groups * rows < 2^30.
 */
dg_status dg_quantize_fp4(const void* x, int x_type, void* q, uint32_t* sf,
                          int groups, int rows, int k, void* stream);
dg_status dg_dequantize_fp4(const void* q, const uint32_t* sf, void* x,
                            int groups, int rows, int k, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_FP4_H */
