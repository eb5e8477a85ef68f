/*
 * agmm_long.h — long contexts over the paged key-value cache of agmm_attn.h on AMD MI355X (gfx950):
 * the C ABI.
 *
 *   ag_prefix_*  attention of one new token of every sequence where sequences share prefixes, which are
 *                read once for every 128 rows (q heads of one kv head) of all that share one;
 *   ag_index_*   an index of the cache's pages, the pages that its score selects for each sequence and kv
 *                head, and (ag_attn_run_heads) the attention over those;
 *   ag_mass_*    the attention weight that each cached token has got, added up step by step;
 *   ag_evict_*   the tokens that such masses keep, and their rows moved together.
 *
 * Types, strides, devices, codes and threading are those of agmm_attn.h. No call here waits for the device;
 * all of them may be captured into a HIP graph and replayed. At most 2^21 sequences times kv heads, but for
 * ag_prefix_run and ag_attn_run_heads, whose limits are ag_attn_run's, and less than 2^31 - 2^20 tokens in a table's
 * pages, but for the own tables of those two. Page numbers and lengths are read on
 * the device and checked there: nothing is read or written at a page outside [0, num_pages).
 */
#ifndef AGMM_LONG_H
#define AGMM_LONG_H

#include "agmm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- shared prefixes ----
 * The sequences of a batch come in groups, runs of neighbours: sequence b is in group g if starts[g] <= b
 * < starts[g + 1]. Its tokens are the first prefix_lens[g] of the group's prefix and then its own, and its new
 * token attends to all of them, as in ag_attn_run. A sequence outside of all groups has its own tokens
 * alone. The prefixes' tokens and the own ones lie in one cache.
 * Two launches: all rows of a group (its sequences' q heads of one kv head) against the prefix and, beside them, the
 * own tokens, in pieces that go to `scratch`; and then the pieces joined, in a fixed order. Results do not depend on
 * timing. */

/* Device bytes of a run's scratch, or a negative code. Host only. It has a piece for each workgroup that the chip holds,
 * whatever the lengths: 17 MB for heads of up to 64 and 34 above, and 8 bytes for each element of a row. */
int64_t ag_prefix_scratch_bytes(const ag_attn_desc* desc, int64_t batch, int64_t groups);

/* One run of a handle of ag_attn_create whose desc has no window, and a cap or a scale of 2^63 at most (else
 * UNSUPPORTED). Scores of 2^127 and more, without a cap, count as infinite.
 *   prefix_table: device int32 [groups], entry (g, j) at g * prefix_row + j, j < prefix_pages;
 *   prefix_lens:  device int32 [groups]; < 0 counts as 0, tokens past the table are left out;
 *   starts:       device int32 [groups + 1], or NULL with one group: all of the batch. Numbers outside [0,
 *                 batch] count as its ends, one below the largest before it as that;
 *   scratch:      device, 256-byte aligned, at least ag_prefix_scratch_bytes(desc, batch, groups); holds
 *                 nothing from one run to the next, and one run at a time may use it.
 *   The rest as for ag_attn_run, lens counting own tokens alone.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED, WRONG_DEVICE or HIP. */
int ag_prefix_run(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                  int64_t q_head, const int32_t* prefix_table, int64_t prefix_row, int64_t prefix_pages,
                  const int32_t* prefix_lens, const int32_t* starts, int64_t groups,
                  const int32_t* page_table, int64_t table_row, int64_t table_len, const int32_t* lens,
                  int64_t batch, void* out, int64_t o_batch, int64_t o_head, float* lse, void* scratch,
                  int64_t scratch_bytes, void* hip_stream);

/* ---- pages selected by a cheap score ----
 * The index holds, for every page and kv head, 2 * head_dim codes (int8) and a scale byte: with e the least
 * whole number from -126 on for which max |k| <= 127 * 2^e over the page's keys (the values that are
 * attended to, of the tokens that count), the scale byte is e + 127, code d is the least whole number >= max_t
 * k_td / 2^e and code head_dim + d the largest <= min_t k_td / 2^e. A page whose keys have a NaN or an infinity
 * gets scale byte 255.
 * The score of a page for a sequence's kv head: with f the least whole number from -126 on for which max
 * |q| <= 127 * 2^f over the head's q heads, and c_hd = q_hd / 2^f rounded to nearest, ties to even,
 *     score = float(sum_hd (c_hd > 0 ? c_hd * code d : c_hd * code (head_dim + d))) * 2^e
 * in 32-bit arithmetic: what the heads' q . k adds up to at most, in the codes. The sum is one of whole numbers,
 * so no order of summation changes it. Elements of q that are not finite count as 0. A page with scale byte 255
 * comes before all others. */
typedef struct ag_page_index {
  int8_t* codes;       /* device [num_pages][kv_heads][2 * head_dim], 16-byte aligned */
  uint8_t* scales;     /* device [num_pages][kv_heads] */
} ag_page_index;

/* Makes the entries of the pages that hold tokens [starts[b], lens[b]) of each sequence, from all of a page's
 * tokens below lens[b].
 *   page_table, table_row, table_len, lens: as for ag_attn_run;
 *   starts: device int32 [batch], < 0 counts as 0; NULL: 0 for all.
 * Absent pages are left out. A page in several of the places that are renewed gets the entry of the one with the most of
 * its tokens; places in front of starts[b] do not count. (To find that, a sequence that ends inside a page reads the
 * numbers of all pages that the call renews.)
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_index_update(const ag_kv_cache* cache, const ag_page_index* index, const int32_t* page_table,
                    int64_t table_row, int64_t table_len, const int32_t* starts, const int32_t* lens,
                    int64_t batch, void* hip_stream);

/* Device bytes of ag_index_select's scratch. Host only. */
int64_t ag_index_scratch_bytes(const ag_kv_cache* cache, int64_t table_len, int64_t batch);

/* The pages that each sequence's new token attends to, for each kv head: of the pages with tokens below
 * lens[b] that are not absent the first `sink` of the table, the last `recent`, and of the others those with the
 * highest scores (the earlier where they are equal), `budget` in all, or all where there are no more.
 *   q: as for ag_attn_run, q_heads heads;
 *   out_table: device int32 [batch][kv_heads][budget]: the selected pages in the order of the tokens, then -1;
 *   out_lens: device int32 [batch]: the tokens in them.
 *   scratch: device, 16-byte aligned, as for ag_prefix_run.
 * sink >= 0, recent >= 1, sink + recent <= budget. At most 128 q heads for a kv head.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_index_select(const ag_kv_cache* cache, const ag_page_index* index, const void* q, int64_t q_batch,
                    int64_t q_head, int64_t q_heads, const int32_t* page_table, int64_t table_row,
                    int64_t table_len, const int32_t* lens, int64_t batch, int64_t budget, int64_t sink,
                    int64_t recent, int32_t* out_table, int32_t* out_lens, void* scratch,
                    int64_t scratch_bytes, void* hip_stream);

/* As ag_attn_run with a page table for each kv head: entry (b, h, j) at b * table_row + h * table_head + j. */
int ag_attn_run_heads(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                      int64_t q_head, const int32_t* page_table, int64_t table_row, int64_t table_head,
                      int64_t table_len, const int32_t* lens, int64_t batch, void* out, int64_t o_batch,
                      int64_t o_head, float* lse, void* hip_stream);

/* ---- eviction by accumulated attention weight ----
 * Weights come from the new tokens of ag_attn_run over one page table for all heads: not from a prompt's own q, behind
 * a shared prefix or over selected pages. */

/* For every sequence b, kv head h and token t < lens[b]:
 *     out[b][h][t] = decay * mass[b][h][t] + sum over h's q heads of exp(s_t - lse)
 * with the scores s_t of ag_attn_run (desc's scale, window and cap; nothing is added to tokens outside of the
 * window, of absent pages or past the table) and its lse. lse = -infinity adds nothing. Entries from lens[b] on are
 * copied, so out may be mass itself (with its strides) but may not overlap it otherwise.
 *   desc: as for ag_attn_create (num_wgs is not used). q, page_table, lens: as for ag_attn_run.
 *   lse: device float [batch][q_heads];
 *   mass, out: device float, entry (b, h, t) at b * batch + h * head + t of the given strides, t < tokens.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_mass_add(const ag_attn_desc* desc, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                int64_t q_head, const float* lse, const int32_t* page_table, int64_t table_row,
                int64_t table_len, const int32_t* lens, int64_t batch, const float* mass,
                int64_t mass_batch, int64_t mass_head, float* out, int64_t out_batch, int64_t out_head,
                int64_t tokens, float decay, void* hip_stream);

/* The tokens that each sequence keeps for each kv head, of those below lens[b] and `tokens` whose pages are not
 * absent: the first `sink` of the sequence, the last `recent`, and of the others those with the most mass (the
 * earlier where they are equal; NaN is the most), `budget` in all, or all where there are no more.
 *   mass: as above;
 *   kept: device int32 [batch][kv_heads][budget]: the tokens in ascending order, then -1;
 *   out_mass: device float [batch][kv_heads][budget]: their masses, then 0; NULL: not wanted;
 *   out_lens: device int32 [batch]: how many they are.
 * sink >= 0, recent >= 0, sink + recent <= budget.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_evict_choose(const ag_kv_cache* cache, const float* mass, int64_t mass_batch, int64_t mass_head,
                    int64_t tokens, const int32_t* page_table, int64_t table_row, int64_t table_len,
                    const int32_t* lens, int64_t batch, int64_t budget, int64_t sink, int64_t recent,
                    int32_t* kept, float* out_mass, int32_t* out_lens, void* hip_stream);

/* Moves kept tokens' rows together: row j of sequence b and kv head h in `to` is set to the row of token
 * kept[b][h][j] in `from`, for j < lens[b] and j < budget, keys, values and scales. Rows whose page is absent, in
 * either table, are left as they are. The two caches have one dtype, storage, head_dim and kv_heads; no page may be
 * both read and written. A row that is written twice (a page in several places of to_table) is left undefined.
 *   kept: as above; lens: device int32 [batch].
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_evict_move(const ag_kv_cache* from, const int32_t* from_table, int64_t from_row, int64_t from_len,
                  const ag_kv_cache* to, const int32_t* to_table, int64_t to_row, int64_t to_len,
                  const int32_t* kept, int64_t budget, const int32_t* lens, int64_t batch,
                  void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* AGMM_LONG_H */
