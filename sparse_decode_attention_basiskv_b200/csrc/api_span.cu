// Entry points of basiskv_cache4.h and basiskv_window.h: argument checks
// (host arithmetic, before any CUDA call) and launch sequences.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/basiskv_cache4.h"
#include "../../include/basiskv_window.h"
#include "cache4.cuh"
#include "internal.h"
#include "launch.cuh"

using namespace basiskv;

// Rounds of the SMs take whole items while they are full.  What is left over is
// cut where that pays: a run costs its KV tiles and about 5 tiles' time for its start
// and end (measured: 16,000 and 3,500 clocks at d 128, r_v 64), the join about 2
// tiles' time and, for writing and reading a run's partials, (r_v + 2) / 6200; a run
// keeps 4 tiles at least, and there are 4 runs an SM at most, which bounds the
// workspace.  Whole / as cut here, us, bf16 r_v 64, r_v 128, 4 bits r_v 64, r_v 128:
// 56 items over 16K tokens (5 runs each) 309 / 149, 408 / 196, 289 / 138, 328 / 163;
// 24 over 4K (6) 80 / 32, 104 / 38, 72 / 30, 76 / 33; 8 over 32K (16) 578 / 59, 923 / 75,
// 516 / 53, 547 / 58.  128 items stay whole: in 8 runs each, 37,000 tokens take 690
// for 696, 960 for 903, 602 for 597, 714 for 684.
TcPlan basiskv::tc_plan(int B, int Hkv, int G, int n_tot, int max_seq_len, int sink, int window,
                        int r_v) {
  const int sms = num_sms(), tq2 = 256 / G;
  const long long items = (long long)B * Hkv * ((n_tot + tq2 - 1) / tq2);
  TcPlan p{(int)(items / sms * sms), (int)(items % sms), 1};
  if (p.tail == 0) return p;
  long long span = max_seq_len;
  if (window > 0 && (long long)window + tq2 + sink < span) span = (long long)window + tq2 + sink;
  const long long tiles = (span + 127) / 128 + 1;
  long long best = -1;  // in hundredths of a tile's time
  for (int ns = 1; ns <= 64 && (ns == 1 || (tiles / ns >= 4 && p.tail * ns <= kTcMaxRuns * sms));
       ++ns) {
    const long long runs = (long long)p.tail * ns, rounds = (runs + sms - 1) / sms;
    long long cost = 100 * rounds * ((tiles + ns - 1) / ns + 5);
    if (ns > 1) cost += 200 + runs * (r_v + 2) / 62;
    if (best < 0 || cost < best) {
      best = cost;
      p.ns = ns;
    }
  }
  return p;
}

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define BKV_NEED(p, n)                                          \
  do {                                                          \
    if (!(p) || !aligned(p, n)) return BASISKV_ERR_INVALID_ARG; \
  } while (0)
#define BKV_MAY(p, n)                                          \
  do {                                                         \
    if ((p) && !aligned(p, n)) return BASISKV_ERR_INVALID_ARG; \
  } while (0)

int status_of(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? BASISKV_OK : BASISKV_ERR_LAUNCH_FAILED;
}

int check_cache4(const basiskv_dims* d) {
  const int rc = validate_dims(d);
  if (rc) return rc;
  if (d->page_size != 16 && d->page_size != 32) return BASISKV_ERR_UNSUPPORTED_SHAPE;
  if (d->cache_fp8) return BASISKV_ERR_INVALID_ARG;  // one element type
  if ((d->route_page && d->route_page != d->page_size) ||
      (d->route_r_v && d->route_r_v != d->r_v) || (d->route_r_k && d->route_r_k != d->r_k))
    return BASISKV_ERR_UNSUPPORTED_SHAPE;
  return BASISKV_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 256)) return BASISKV_ERR_INVALID_ARG;
  return have < need ? BASISKV_ERR_WORKSPACE_TOO_SMALL : BASISKV_OK;
}

// The arguments every attention over spans shares.
SpanArgs span_args(const basiskv_dims* d, const basiskv_bf16* q, const int32_t* seq_lens,
                   int max_seq_len, const int32_t* block_table, const void* K, const void* Z,
                   basiskv_bf16* out, unsigned int* status) {
  SpanArgs a{};
  a.q = q;
  a.K = static_cast<const uint8_t*>(K);
  a.Z = static_cast<const uint8_t*>(Z);
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.out = out;
  a.B = d->B;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.G = d->Hq / d->Hkv;  // 1, 2, 4 or 8
  a.logG = a.G == 8 ? 3 : a.G >> 1;
  a.d = d->d;
  a.r_v = d->r_v;
  a.S = d->page_size;
  a.logS = d->page_size == 8 ? 3 : (d->page_size == 16 ? 4 : 5);
  a.max_pages = d->max_pages_per_seq;
  a.num_phys = d->num_phys_pages;
  a.max_seq_len = max_seq_len;
  a.zsplit = d->route_r_v ? d->route_r_v : d->r_v;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d->d));
  a.status = status;
  return a;
}

size_t span_partial_bytes(const basiskv_dims* d, int rows) {
  return (span_slots(d->B, d->Hkv) * rows * (d->r_v + kSpanRowPad) * 4 + 255) & ~size_t(255);
}

int check_window(const basiskv_dims* d, int n_q, int max_seq_len, int sink, int window) {
  if (!d || (d->cache_fp8 != 0 && d->cache_fp8 != 1)) return BASISKV_ERR_INVALID_ARG;
  basiskv_dims plain = *d;  // the E4M3 router's and the routing page's limits do not apply
  plain.cache_fp8 = 0;
  plain.route_page = 0;
  const int rc = validate_dims(&plain);
  if (rc) return rc;
  const long long cap = (long long)d->max_pages_per_seq * d->page_size;
  if (max_seq_len < 1 || max_seq_len > cap || n_q < 1 || n_q > cap || sink < 0 || window < 0)
    return BASISKV_ERR_INVALID_ARG;
  return BASISKV_OK;
}

// The mask with bounds that cover the whole context written as such.
struct Mask {
  int sink, window;
};
Mask window_mask(int max_seq_len, int sink, int window) {
  return {sink < max_seq_len ? sink : max_seq_len, window < max_seq_len ? window : 0};
}

// Which calls are streamed, by the rows (query tokens times group heads) that share a
// Key and by the tokens of all heads that the call may read; the others go to the
// tensor cores, whose tiles hold 128 rows.
//
// Always up to 16 rows.  17 to 24 rows from 128K tokens on, 25 to 32 from 256K (r_v
// 128: 384K; over bf16 caches with r_v above 64 never): there a lane's queries and
// accumulators fill its registers.  Both sides, streamed / tensor cores, us, captured
// calls, d 128, r_v 64 unless said:
//   16 rows, 64K tokens (1 x 8 heads)  bf16 18.6 / 22.3   E4M3 17.8 / 23.3   4 bits 17.4 / 21.7
//   24 rows, 64K                       bf16 25.4 / 22.9   E4M3 24.0 / 24.3   4 bits 25.2 / 22.3
//            128K                      bf16 30.4 / 30.9   E4M3 27.2 / 31.3   4 bits 28.1 / 28.9
//            448K (7 x 8 heads)        bf16 51.1 / 68.0   E4M3 38.5 / 79.2   4 bits 37.5 / 71.6
//   32 rows, 128K                      bf16 35.0 / 30.0   E4M3 31.8 / 31.3   4 bits 33.0 / 28.9
//            256K                      bf16 47.2 / 44.6   E4M3 39.6 / 48.5   4 bits 40.1 / 41.5
//            448K                      bf16 61.3 / 68.3   E4M3 46.1 / 79.5   4 bits 45.5 / 71.2
//   32 rows, r_v 128, 256K             bf16 69.5 / 52.6   E4M3 63.4 / 72.5   4 bits 59.2 / 48.0
//            448K                      bf16 93.8 / 86.8   E4M3 78.1 / 128    4 bits 75.1 / 85.2
//            1M                        bf16 184 / 158     E4M3 147 / 243     4 bits 142 / 159
//   32 rows, r_v 96, 1M                bf16 173 / 146     E4M3 98 / 171      4 bits 96 / 151
bool window_streams(const basiskv_dims* d, int n_q, int max_seq_len, Mask m, bool cache4) {
  const int G = d->Hq / d->Hkv;
  if (n_q <= 16 / G) return true;
  if (n_q > kSpanMaxRows / G) return false;
  if (d->cache_fp8 && d->page_size < 16) return false;  // two pages of 16 make a unit there
  const long long seen = (long long)m.window + n_q + m.sink;
  const long long span = m.window > 0 && seen < max_seq_len ? seen : max_seq_len;
  const long long tokens = span * d->B * d->Hkv;
  if (n_q <= 24 / G) return tokens >= 128 << 10;
  if (!d->cache_fp8 && !cache4 && d->r_v > 64) return false;
  return tokens >= (d->r_v == 128 ? 384 : 256) << 10;
}

size_t window_bytes(const basiskv_dims* d, int n_q, int max_seq_len, int sink, int window) {
  const int G = d->Hq / d->Hkv;
  const Mask m = window_mask(max_seq_len, sink, window);
  // (which caches the call will have, bf16 or 4 bits, is not known here)
  const bool any = window_streams(d, n_q, max_seq_len, m, true);
  const size_t streamed = any ? span_partial_bytes(d, n_q * G) : 256;
  if (any && window_streams(d, n_q, max_seq_len, m, false)) return streamed;
  const TcPlan plan = tc_plan(d->B, d->Hkv, G, n_q, max_seq_len, m.sink, m.window, d->r_v);
  const size_t n = tc_partial_bytes(plan, d->r_v);
  return n > streamed ? (n + 255) & ~size_t(255) : streamed;
}

}  // namespace

extern "C" {

size_t basiskv_cache4_bytes(const basiskv_dims* dims, int width) {
  if (check_cache4(dims) != BASISKV_OK) return 0;
  if (width != dims->d && width != dims->r_v && width != dims->r_k) return 0;
  return (size_t)dims->num_phys_pages * dims->Hkv * q4_tile_bytes(dims->page_size, width);
}

int basiskv_cache4_write(const basiskv_dims* dims, const basiskv_bf16* k_new,
                         const basiskv_bf16* z_new, const basiskv_bf16* e_new, int n_new,
                         const int32_t* seq_lens, int32_t* lens_out, const int32_t* block_table,
                         uint8_t* K4, uint8_t* Z4, uint8_t* E4, void* stream) {
  int rc = check_cache4(dims);
  if (rc) return rc;
  if (n_new < 1 || (long long)n_new > (long long)dims->max_pages_per_seq * dims->page_size)
    return BASISKV_ERR_INVALID_ARG;
  BKV_NEED(k_new, 16);
  BKV_NEED(z_new, 16);
  BKV_NEED(K4, 16);
  BKV_NEED(Z4, 16);
  if (!e_new != !E4) return BASISKV_ERR_INVALID_ARG;
  BKV_MAY(e_new, 16);
  BKV_MAY(E4, 16);
  BKV_NEED(seq_lens, 4);
  BKV_MAY(lens_out, 4);
  BKV_NEED(block_table, 4);
  Cache4Args a{};
  a.status = device_status_ptr();
  if (!a.status) return BASISKV_ERR_CUDA;
  a.rows[0] = k_new, a.rows[1] = z_new, a.rows[2] = e_new;
  a.cache[0] = K4, a.cache[1] = Z4, a.cache[2] = E4;
  a.width[0] = dims->d, a.width[1] = dims->r_v, a.width[2] = dims->r_k;
  for (int i = 0; i < 3; ++i) a.blocks[i] = a.rows[i] ? dims->Hkv * a.width[i] / 16 : 0;
  a.seq_lens = seq_lens;
  const bool in_place = lens_out == seq_lens;
  a.lens_out = in_place ? nullptr : lens_out;
  a.block_table = block_table;
  a.B = dims->B, a.n = n_new, a.Hkv = dims->Hkv, a.S = dims->page_size;
  a.logS = dims->page_size == 16 ? 4 : 5;
  a.max_pages = dims->max_pages_per_seq, a.num_phys = dims->num_phys_pages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = status_of(launch_cache4_write(a, st, pdl_allowed()));
  if (rc || !in_place) return rc;
  // in place, the lengths move only once every CTA has read them
  AppendArgs b{};
  b.seq_lens = seq_lens;
  b.seq_lens_out = lens_out;
  b.B = dims->B, b.n_new = n_new, b.max_pages = dims->max_pages_per_seq, b.S = dims->page_size;
  b.status = a.status;
  return status_of(launch_bump_lengths(b, st, pdl_allowed()));
}

int basiskv_cache4_read(const basiskv_dims* dims, const int32_t* first, int count,
                        const int32_t* seq_lens, const int32_t* block_table, const uint8_t* K4,
                        const uint8_t* Z4, const uint8_t* E4, basiskv_bf16* k_out,
                        basiskv_bf16* z_out, basiskv_bf16* e_out, void* stream) {
  int rc = check_cache4(dims);
  if (rc) return rc;
  if (count < 1 || (long long)count > (long long)dims->max_pages_per_seq * dims->page_size)
    return BASISKV_ERR_INVALID_ARG;
  BKV_NEED(first, 4);
  BKV_NEED(seq_lens, 4);
  BKV_NEED(block_table, 4);
  if (!k_out != !K4 || !z_out != !Z4 || !e_out != !E4 || (!k_out && !z_out && !e_out))
    return BASISKV_ERR_INVALID_ARG;
  BKV_MAY(K4, 16);
  BKV_MAY(Z4, 16);
  BKV_MAY(E4, 16);
  BKV_MAY(k_out, 16);
  BKV_MAY(z_out, 16);
  BKV_MAY(e_out, 16);
  Cache4Args a{};
  a.status = device_status_ptr();
  if (!a.status) return BASISKV_ERR_CUDA;
  a.out[0] = k_out, a.out[1] = z_out, a.out[2] = e_out;
  a.cache[0] = const_cast<uint8_t*>(K4);
  a.cache[1] = const_cast<uint8_t*>(Z4);
  a.cache[2] = const_cast<uint8_t*>(E4);
  a.width[0] = dims->d, a.width[1] = dims->r_v, a.width[2] = dims->r_k;
  for (int i = 0; i < 3; ++i) a.blocks[i] = a.out[i] ? dims->Hkv * a.width[i] / 16 : 0;
  a.first = first;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.B = dims->B, a.n = count, a.Hkv = dims->Hkv, a.S = dims->page_size;
  a.logS = dims->page_size == 16 ? 4 : 5;
  a.max_pages = dims->max_pages_per_seq, a.num_phys = dims->num_phys_pages;
  return status_of(launch_cache4_read(a, static_cast<cudaStream_t>(stream), pdl_allowed()));
}

int basiskv_cache4_route(const basiskv_dims* dims, const basiskv_bf16* q, const int32_t* seq_lens,
                         int max_seq_len, const int32_t* block_table, const basiskv_bf16* P_K,
                         const basiskv_bf16* U_K, const uint8_t* Z4, const uint8_t* E4, int top_k,
                         float* page_scores, int32_t* sel, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int rc = check_cache4(dims);
  if (rc) return rc;
  rc = validate_len_topk(dims, top_k, max_seq_len);
  if (rc) return rc;
  BKV_NEED(q, 16);
  BKV_NEED(seq_lens, 4);
  BKV_NEED(block_table, 4);
  BKV_NEED(P_K, 16);
  BKV_NEED(U_K, 16);
  BKV_NEED(Z4, 16);
  BKV_NEED(E4, 16);
  if (!sel && !page_scores) return BASISKV_ERR_INVALID_ARG;  // nothing to write
  BKV_MAY(sel, 4);
  BKV_MAY(page_scores, 4);
  const WsRegions L = workspace_regions(dims, top_k);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool pdl = pdl_allowed();
  unsigned int* status = device_status_ptr();
  if (!status) return BASISKV_ERR_CUDA;
  float* qt = reinterpret_cast<float*>(ws + L.qt);
  FoldQArgs f{q, P_K, U_K, qt, dims->B, dims->Hq, dims->Hkv, dims->d, dims->r_v, dims->r_k};
  rc = status_of(launch_fold_query(f, st, pdl));
  if (rc) return rc;
  Route4Args r{};
  r.qt = qt;
  r.Z = Z4;
  r.E = E4;
  r.seq_lens = seq_lens;
  r.block_table = block_table;
  r.scores = page_scores ? page_scores : reinterpret_cast<float*>(ws + L.scores);
  r.B = dims->B, r.Hq = dims->Hq, r.Hkv = dims->Hkv, r.G = dims->Hq / dims->Hkv;
  r.r_v = dims->r_v, r.r_k = dims->r_k, r.S = dims->page_size;
  r.max_pages = dims->max_pages_per_seq, r.num_phys = dims->num_phys_pages;
  r.max_seq_len = max_seq_len;
  r.status = status;
  rc = status_of(launch_route4(r, st, pdl));
  if (rc || !sel) return rc;
  const int n_sink = dims->sink_pages == 0 ? 1 : (dims->sink_pages < 0 ? 0 : dims->sink_pages);
  SelectArgs s{r.scores, seq_lens, sel, dims->B, dims->Hkv, dims->page_size,
               dims->max_pages_per_seq, top_k, max_seq_len, 0, block_table,
               reinterpret_cast<int32_t*>(ws + L.selp), n_sink,
               dims->recent_pages == 0 ? 1 : dims->recent_pages, 1, 1};
  return status_of(launch_select(s, st, pdl));
}

int basiskv_cache4_attend(const basiskv_dims* dims, const basiskv_bf16* q,
                          const int32_t* seq_lens, int max_seq_len, const int32_t* block_table,
                          const uint8_t* K4, const uint8_t* Z4, const int32_t* sel, int top_k,
                          basiskv_bf16* a_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int rc = check_cache4(dims);
  if (rc) return rc;
  rc = validate_len_topk(dims, top_k, max_seq_len);
  if (rc) return rc;
  BKV_NEED(q, 16);
  BKV_NEED(seq_lens, 4);
  BKV_NEED(block_table, 4);
  BKV_NEED(K4, 16);
  BKV_NEED(Z4, 16);
  BKV_NEED(sel, 4);
  BKV_NEED(a_out, 16);
  const WsRegions L = workspace_regions(dims, top_k);
  rc = check_workspace(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  unsigned int* status = device_status_ptr();
  if (!status) return BASISKV_ERR_CUDA;
  SpanArgs a = span_args(dims, q, seq_lens, max_seq_len, block_table, K4, Z4, a_out, status);
  a.sel = sel;
  a.top_k = top_k;
  a.n_tot = 1;
  // With N = B * Hkv the workspace holds (1024 + N) G (r_v + 2) partials and, behind
  // them, N G r_v sums of the sparse decode, which this call does not make: more
  // than the (kSpanMaxCtas + N) G (r_v + kSpanRowPad) floats that are written.
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.partial);
  return status_of(launch_span_q4(a, static_cast<cudaStream_t>(stream), pdl_allowed()));
}

size_t basiskv_window_workspace_size(const basiskv_dims* dims, int n_q, int max_seq_len,
                                     int sink_tokens, int window) {
  if (check_window(dims, n_q, max_seq_len, sink_tokens, window) != BASISKV_OK) return 0;
  return window_bytes(dims, n_q, max_seq_len, sink_tokens, window);
}

int basiskv_attend_window(const basiskv_dims* dims, const basiskv_bf16* q, int n_q,
                          const int32_t* seq_lens, int max_seq_len, const int32_t* block_table,
                          const void* K_cache, const void* Z_cache, int cache4, int sink_tokens,
                          int window, basiskv_bf16* a_out, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = check_window(dims, n_q, max_seq_len, sink_tokens, window);
  if (rc) return rc;
  if (cache4 != 0 && cache4 != 1) return BASISKV_ERR_INVALID_ARG;
  if (cache4) {
    rc = check_cache4(dims);
    if (rc) return rc;
  }
  BKV_NEED(q, 16);
  BKV_NEED(seq_lens, 4);
  BKV_NEED(block_table, 4);
  BKV_NEED(K_cache, 16);
  BKV_NEED(Z_cache, 16);
  BKV_NEED(a_out, 16);
  rc = check_workspace(workspace, workspace_bytes,
                       window_bytes(dims, n_q, max_seq_len, sink_tokens, window));
  if (rc) return rc;
  unsigned int* status = device_status_ptr();
  if (!status) return BASISKV_ERR_CUDA;
  SpanArgs a = span_args(dims, q, seq_lens, max_seq_len, block_table, K_cache, Z_cache, a_out,
                         status);
  const Mask m = window_mask(max_seq_len, sink_tokens, window);
  a.sink = m.sink;
  a.window = m.window;
  a.partial = static_cast<float*>(workspace);
  a.n_tot = n_q;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool pdl = pdl_allowed();
  if (window_streams(dims, n_q, max_seq_len, m, cache4))
    return status_of(cache4 ? launch_span_q4(a, st, pdl)
                            : dims->cache_fp8 ? launch_span_e4m3(a, st, pdl)
                                              : launch_span_bf16(a, st, pdl));
  return status_of(cache4 ? launch_span_tc_q4(a, st, pdl)
                          : dims->cache_fp8 ? launch_span_tc_e4m3(a, st, pdl)
                                            : launch_span_tc_bf16(a, st, pdl));
}

}  // extern "C"
