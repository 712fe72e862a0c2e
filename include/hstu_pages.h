/*
 * hstu_pages.h -- paged history of the HSTU stack: writing rows into pages
 * (quantised as they are written), reading them back, and the attention and
 * the stack step of new actions and M-FALCON candidates over pages.  Part of
 * libhstu.so; the conventions of hstu.h hold for every entry point.
 */
#ifndef HSTU_B200_PAGES_H_
#define HSTU_B200_PAGES_H_

#include "hstu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Paged history ----
 * A history cache whose users grow by single actions, come and go: the keys
 * and values of a layer (SiLU(f1(.)) of the history rows, as in the history
 * cache of hstu.h) live in pages of page_size rows, and a page table says which
 * pages are a user's.  Position j of user b (its local index, 0 = oldest) is
 * row j % page_size of page page_table[b * table_width + j / page_size].  The
 * caller owns the pools, the page table and the lengths, and gives pages out;
 * the library reads and writes them.  What a new action needs is then its own
 * rows and its user's pages: nothing is computed again or copied when a user's
 * history grows, and the pages of a user who left serve another.
 *
 * Formats: BF16 and FP32 hold the rows as they are.  E4M3 holds a block (one
 * head's key or value of one row) as 8-bit codes and one scale byte:
 *   m      = max |x_i| over the finite x_i of the block
 *   e      = the smallest integer with m <= 448 * 2^e, held in [-126, 120]; 0 if m = 0
 *   code_i = x_i * 2^-e rounded to the nearest e4m3 (ties to even), held to
 *            +-448 (+-240 at e = 120, so that code * 2^e is finite);
 *            an infinity or a NaN becomes NaN
 *   scale  = e + 127
 * and reads back as code_i * 2^e, exactly.  BF16 compute: BF16 or E4M3 pages;
 * FP32 compute: FP32 pages (else HSTU_ERR_UNSUPPORTED). */
typedef enum { HSTU_PAGES_BF16 = 0, HSTU_PAGES_FP32 = 1, HSTU_PAGES_E4M3 = 2 } hstu_page_format;

/* The pages of one layer; device pointers, caller-owned, 16-byte aligned. */
typedef struct {
  hstu_page_format format;
  int32_t page_size;     /* rows of a page: 16, 32, 64, 128 or 256 */
  int32_t num_pages;     /* >= 1; num_pages * num_heads * 2 * page_size < 2^31 */
  void* kv;              /* [num_pages, num_heads, 2, page_size, head_dim]: plane 0 K, plane 1 V */
  uint8_t* scales;       /* E4M3: [num_pages, num_heads, 2, page_size]; else ignored */
  int64_t* timestamps;   /* [num_pages, page_size]; the layers of a stack may share one */
} hstu_page_pool;

/* Arguments that the calls below share:
 *   total_rows   R, 0 <= R <= max_tokens: rows of the call's [R, *] tensors
 *   seq_offsets  device int32 [num_users + 1], 0 = offsets[0] <= ... <= offsets[B] <= R:
 *                user b owns rows offsets[b] .. offsets[b+1]-1 (none is allowed).  Rows from
 *                offsets[B] on (the padding of a launch of fixed size) have to be readable,
 *                but their values reach nothing, and their outputs are left as they were
 *   page_table   device int32 [num_users, table_width]; entries that no position of the call
 *                needs are not read.  table_width * page_size <= 2^30
 * The calls work on the rows, pages and tables as they are in stream order, so
 * a captured call follows the lengths and tables of each replay.  A page that
 * two users share may be read by both; positions that one call writes must be
 * distinct.  Device-side findings set HSTU_DEVERR_OFFSETS, _PAGES or
 * _TIMESTAMPS in the handle's error word; the user or row they concern is
 * skipped and its outputs are undefined (offsets that fall or leave the rows
 * concern every user: the attention then writes nothing).
 *
 * The attention uses the handle's workspace (32 KB an SM in every handle, 4.8 MB on a
 * B200): the calls of one handle, and the replays of its captured calls, must not
 * overlap.  Its waits are bounded as hstu_set_wait_limit says; one that expires sets
 * HSTU_DEVERR_TIMEOUT, and the handle's attention over pages is undefined until
 * hstu_get_device_error has been called.  Infinities and NaN among the q, k and v of a row
 * or the keys and values it sees make its outputs of that head non-finite or NaN, not more;
 * so do finite ones with a score, or (E4M3) a SiLU(score) * 2^e of a value's block, that
 * fp32 does not hold. */

/* Writes (and quantises) rows into pages: row offsets[b] + i of `uvqk` becomes
 * position start[b] + i of user b.
 *   uvqk         device [R, 4d] compute dtype: columns U | V | Q | K (V and K are read)
 *   timestamps   device int64 [R], written beside the rows, or NULL: the pages' timestamps
 *                stay (another layer's call has written the shared ones)
 *   start        device int32 [num_users], or NULL: every user from position 0 */
hstu_status hstu_pages_write(hstu_handle* h, const hstu_page_pool* pool, const void* uvqk,
                             int64_t total_rows, const int32_t* seq_offsets, int32_t num_users,
                             const int64_t* timestamps, const int32_t* page_table,
                             int32_t table_width, const int32_t* start, void* stream);

/* Reads rows back: position start[b] + i of user b becomes row offsets[b] + i.
 *   uvqk         device [R, 4d] compute dtype: the V and K columns are written (e4m3 pages:
 *                code * 2^e, exact in bf16), the U and Q columns left as they were
 *   timestamps   device int64 [R] (written) or NULL */
hstu_status hstu_pages_read(hstu_handle* h, const hstu_page_pool* pool, const int32_t* page_table,
                            int32_t table_width, const int32_t* start, const int32_t* seq_offsets,
                            int32_t num_users, int64_t total_rows, void* uvqk,
                            int64_t* timestamps, void* stream);

/* Equation (2) for new rows over their users' pages: with n = lengths[b], row r
 * of user b (a new action, or an M-FALCON candidate: the same case) sits at
 * position n and sees the positions 0 .. n - 1 of the pages and itself,
 *   s_j = q_r . k_j + rab_pos[min(n - j, pos_clamp)] + rab_time[t(ts_r - ts_j)]
 *   s_r = q_r . k_r + rab_pos[0] + rab_time[0]
 *   av[r, h-th head] = (sum_j SiLU(s_j) v_j + SiLU(s_r) v_r) / n_norm
 * with k_r, v_r from the row itself, so the result does not depend on whether
 * the row has been written to a page.  Made for one or a few rows a user, and
 * takes more rows of a user at once where R > num_users: leave users without rows
 * out of a call for several rows of a few.  The history is split over the GPU and
 * the parts are joined in a fixed order, so a call gives the same bits every time.
 *   uvqk         device [R, 4d] compute dtype (V, Q and K are read)
 *   timestamps   device int64 [R], in [0, 2^62)
 *   lengths      device int32 [num_users]: cached rows of each user, >= 0
 *   rab_pos, rab_time   as in hstu_layer_weights
 *   av           device fp32 [R, d]
 * Needs a fixed n_norm (> 0), as the history cache does, and
 * R * num_heads * (table_width * page_size / 64 + 1) <= 2^30; else HSTU_ERR_UNSUPPORTED. */
hstu_status hstu_pages_attention(hstu_handle* h, const hstu_page_pool* pool, const void* uvqk,
                                 int64_t total_rows, const int32_t* seq_offsets,
                                 int32_t num_users, const int64_t* timestamps,
                                 const int32_t* page_table, int32_t table_width,
                                 const int32_t* lengths, const float* rab_pos,
                                 const float* rab_time, float* av, void* stream);

/* Runs the stack over histories (causal mode) and writes each layer's K and V
 * and the timestamps to the pages, from position 0 of every user.  pools: host
 * array of num_layers pools.  `out` receives the histories' outputs (may alias
 * `values`); here offsets[B] = R.  Other arguments as for hstu_stack_forward. */
hstu_status hstu_pages_prefill(hstu_handle* h, const hstu_page_pool* pools, const void* values,
                               int64_t total_rows, const int32_t* seq_offsets, int32_t num_users,
                               const int64_t* timestamps, const hstu_layer_weights* layers,
                               int32_t num_layers, const int32_t* page_table, int32_t table_width,
                               void* out, void* stream);

/* Runs the stack for new rows against the pages.
 *   append != 0: new actions, at most one row a user: each layer's K and V and
 *                the row's timestamp are written at position lengths[b] (which
 *                its page table row must hold); the caller then raises lengths[b]
 *   append == 0: candidates, any number of rows a user; the pages stay
 *   values       device [R, d] io_dtype;  out  device [R, d] io_dtype, may alias values
 * Rows from offsets[B] on leave undefined rows of `out`. */
hstu_status hstu_pages_step(hstu_handle* h, const hstu_page_pool* pools, const void* values,
                            int64_t total_rows, const int32_t* seq_offsets, int32_t num_users,
                            const int64_t* timestamps, const hstu_layer_weights* layers,
                            int32_t num_layers, const int32_t* page_table, int32_t table_width,
                            const int32_t* lengths, int32_t append, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_B200_PAGES_H_ */
