/*
 * basiskv_window.h — attention over a sliding window and a few first tokens
 * that stay visible (sinks), for single tokens and prompt chunks, over bf16,
 * E4M3 and 4-bit caches.  The conventions of basiskv.h hold.
 */
#ifndef BASISKV_WINDOW_H_
#define BASISKV_WINDOW_H_

#include "basiskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace basiskv_attend_window needs for n_q query tokens per
 * sequence, contexts of at most max_seq_len tokens and this mask; 0 when the
 * arguments are invalid.  It holds for a call with these arguments, whatever the
 * lengths: the work is split otherwise for other ones, and a smaller
 * max_seq_len may need more.  Whatever max_seq_len and the mask, it is at most
 *   (512 + B * Hkv) * R * (r_v + 4) * 4 bytes  for R = n_q * Hq / Hkv <= 16,
 *   4 * SMs * 256 * (r_v + 2) * 4 bytes        for R > 32 (79 MB at r_v 128, 148 SMs),
 * and the larger of the two between, rounded up to 256 bytes. */
BASISKV_API size_t basiskv_window_workspace_size(const basiskv_dims* dims, int n_q,
                                                 int max_seq_len, int sink_tokens, int window);

/* Attention of the last n_q tokens of every sequence (their rows are in the
 * cache already): query token j of sequence b stands at p = seq_lens[b] - n_q + j
 * and, for every query head h of KV head g,
 *   s_t = (q . K_t) / sqrt(d),  a = sum_t softmax(s)_t z_t
 * over the tokens t <= p with t > p - window or t < sink_tokens.
 *   q        bf16 [B][n_q][Hq][d]
 *   window   tokens a query sees up to and including its own; 0 = all
 *   sink_tokens  first tokens that stay visible; 0 = none
 *   cache4   0: K_cache and Z_cache hold bf16, or E4M3 with dims->cache_fp8 = 1;
 *            1: they are 4-bit caches (basiskv_cache4.h; page_size 16 or 32,
 *            dims->cache_fp8 0, no narrow router)
 *   a_out    bf16 [B][n_q][Hq][r_v] (fp32 scores, sums and accumulation, one
 *            rounding; the weights enter the products with 16 significant bits
 *            over bf16 caches and 11 over E4M3 and 4-bit ones, whatever n_q is:
 *            with B * n_q as its batch, the input of basiskv_outproj_sources)
 * Query tokens with p < 0 (n_q past a sequence's length: a batch padded at the
 * front) see nothing; a row that sees nothing is zero.  A sequence whose length
 * is outside [0, max_seq_len] is taken as empty (BASISKV_DEV_BAD_LENGTH).  A
 * block-table entry out of range leaves its page's tokens out
 * (BASISKV_DEV_BAD_PAGE); entries of pages no query sees are not read, so pages
 * that have left the window may be reused.  Cached rows that some query of the
 * call sees must be finite, their latents at most 2^64 in magnitude.
 * dims->route_page, sink_pages and recent_pages are ignored; any page_size of
 * basiskv.h. */
BASISKV_API int basiskv_attend_window(const basiskv_dims* dims, const basiskv_bf16* q, int n_q,
                                      const int32_t* seq_lens, int max_seq_len,
                                      const int32_t* block_table, const void* K_cache,
                                      const void* Z_cache, int cache4, int sink_tokens,
                                      int window, basiskv_bf16* a_out, void* workspace,
                                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BASISKV_WINDOW_H_ */
