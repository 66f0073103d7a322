/*
 * basiskv_cache4.h — 4-bit caches: writing rows, reading them back, page
 * scores and selected attention over them.
 *
 * The conventions of basiskv.h hold (device pointers, streams, host
 * validation before any launch, device status bits, one workspace).  The
 * caches here are a third form of K_cache, Z_cache and E_cache beside bf16
 * and E4M3; dims->cache_fp8, route_page, route_r_v and route_r_k must be 0 (or
 * name the full widths), and page_size 16 or 32.
 *
 * Format.  A row of w columns is cut into blocks of 16.  Every block has one
 * scale byte, 5 exponent bits (bias 15) above 3 mantissa bits: the upper bits
 * of an IEEE half without its sign (half bits = byte << 7).  Every column is
 * an E2M1 code: sign, 2 exponent bits, 1 mantissa bit, the magnitudes 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6.  The cached value is code * scale, exactly, and has at
 * most 6 significant bits (it is a bf16 value and an f16 value).
 *   scale = amax(block) / 6   rounded to 4 significant bits, nearest even
 *           (steps of 2^-17 below 2^-14), at most 10240
 *   code  = x / scale         rounded to E2M1, nearest even, at most +-6
 * Blocks whose scale rounds to 0 hold zeros; |x| above 61440 saturates.  Rows
 * are finite (a NaN is stored as +-6 times its block's scale).
 *   K4, Z4, E4  [num_phys_pages][Hkv] tiles of S * w * 9 / 16 bytes (w = d,
 *               r_v, r_k): codes [S][w / 2], column 2i in the low nibble of
 *               byte i, then scales [S][w / 16].  16-byte aligned.
 * A token and KV head take (d + r_v + r_k) * 9 / 16 bytes, 0.28 of bf16.
 */
#ifndef BASISKV_CACHE4_H_
#define BASISKV_CACHE4_H_

#include "basiskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one 4-bit cache of row width w (d, r_v or r_k) for these dims; 0
 * when the dims are invalid or not supported here. */
BASISKV_API size_t basiskv_cache4_bytes(const basiskv_dims* dims, int width);

/* Writes n_new rows per sequence at tokens seq_lens[b] + j.  z and e rows are
 * the caller's: z = v A_V and e = (k - z P_K) U_K are linear in v and k, so a
 * deployment folds them into the layer's projections.
 *   k_new bf16 [B][n_new][Hkv][d], z_new [..][r_v], e_new [..][r_k]; e_new and
 *   E4 may both be NULL (a layer that is never routed)
 *   seq_lens  int32 [B], the lengths before the call
 *   lens_out  int32 [B] receives seq_lens[b] + n_new; it may be seq_lens itself
 *             (advanced in place, one more launch), or NULL (not written)
 * A sequence whose rows would pass max_pages_per_seq * S is skipped whole:
 * BASISKV_DEV_OVERFLOW is raised and its length stays.  A row whose block-table
 * entry is out of range is skipped (BASISKV_DEV_BAD_PAGE).  Uses no workspace. */
BASISKV_API int basiskv_cache4_write(const basiskv_dims* dims, const basiskv_bf16* k_new,
                                     const basiskv_bf16* z_new, const basiskv_bf16* e_new,
                                     int n_new, const int32_t* seq_lens, int32_t* lens_out,
                                     const int32_t* block_table, uint8_t* K4, uint8_t* Z4,
                                     uint8_t* E4, void* stream);

/* Reads tokens first[b] .. first[b] + count - 1 of every sequence back as the
 * bf16 values they stand for.  Rows of tokens outside [0, seq_lens[b]) are left
 * as they were.
 *   k_out bf16 [B][count][Hkv][d], z_out [..][r_v], e_out [..][r_k]; each of
 *   them may be NULL together with its cache, but not all three
 * Uses no workspace. */
BASISKV_API int basiskv_cache4_read(const basiskv_dims* dims, const int32_t* first, int count,
                                    const int32_t* seq_lens, const int32_t* block_table,
                                    const uint8_t* K4, const uint8_t* Z4, const uint8_t* E4,
                                    basiskv_bf16* k_out, basiskv_bf16* z_out,
                                    basiskv_bf16* e_out, void* stream);

/* basiskv_route over 4-bit caches: the same scores (of the cached values),
 * selection, outputs and errors.  A sequence whose length is outside
 * [0, max_seq_len] is taken as empty (BASISKV_DEV_BAD_LENGTH): it gets no scores,
 * and a selection of -1. */
BASISKV_API int basiskv_cache4_route(const basiskv_dims* dims, const basiskv_bf16* q,
                                     const int32_t* seq_lens, int max_seq_len,
                                     const int32_t* block_table, const basiskv_bf16* P_K,
                                     const basiskv_bf16* U_K, const uint8_t* Z4,
                                     const uint8_t* E4, int top_k, float* page_scores,
                                     int32_t* sel, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* basiskv_attend over 4-bit caches, with the latents written as bf16 [B][Hq][r_v]
 * (fp32 accumulation, one rounding: the input of basiskv_outproj_sources with
 * n_src = 1).  Selected pages past a sequence's length contribute nothing, a page
 * selected twice counts twice; a group without a live selected token gets
 * zeros.  A sequence whose length is outside [0, max_seq_len] is taken as empty
 * (BASISKV_DEV_BAD_LENGTH); basiskv_attend does not check it. */
BASISKV_API int basiskv_cache4_attend(const basiskv_dims* dims, const basiskv_bf16* q,
                                      const int32_t* seq_lens, int max_seq_len,
                                      const int32_t* block_table, const uint8_t* K4,
                                      const uint8_t* Z4, const int32_t* sel, int top_k,
                                      basiskv_bf16* a_out, void* workspace,
                                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BASISKV_CACHE4_H_ */
