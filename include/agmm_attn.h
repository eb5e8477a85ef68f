/*
 * agmm_attn.h — what stands between the two sharded products of an attention block when it
 * serves on AMD MI355X (gfx950): the C ABI.
 *
 * A tensor-parallel attention block enters through the all-gather + GEMM of agmm.h (the fused
 * q/k/v projection, columns split over the ranks) and leaves through its GEMM + all-reduce (the
 * output projection). Between the two each rank needs, for its own heads:
 *
 *   ag_rope_*   rotary positions of q and k, and their gradient;
 *   ag_kv_*     a paged key-value cache: rows written to their slots, quantised on the way if the
 *               cache is stored in 8 or 4 bits, and read back;
 *   ag_attn_*   the attention of one new token of every sequence over that cache.
 *
 * Types: q, k, v and the outputs share one 16-bit type (AGMM_F16 or AGMM_BF16); every sum, angle
 * and softmax statistic is held in 32 bits or more. Strides are counted in elements of the tensor
 * unless they say bytes; a head's values are always contiguous. Kernels are launched on the current
 * device: memory and stream of a call belong to it (handles are checked; the cache's calls have none, and
 * pointers' devices are not looked up). Codes and threading are those of
 * agmm.h (ag_matmul_strerror and ag_matmul_last_hip_error serve these functions too). The
 * creates and destroys wait for the device; the runs, appends and reads do not, and may be captured
 * into a HIP graph and replayed.
 */
#ifndef AGMM_ATTN_H
#define AGMM_ATTN_H

#include "agmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ----
 * For a token at position p, pair i of a head's rotated part turns by the angle p * theta_i:
 *     y1 = magnitude * (x1 * cos - x2 * sin),   y2 = magnitude * (x2 * cos + x1 * sin)
 * and the rest of the head passes through. The gradient is the transposed matrix (angle negated). */
#define AG_ROPE_HALF 0         /* pair i = elements (i, i + rot_dim / 2) of the rotated part */
#define AG_ROPE_INTERLEAVED 1  /* pair i = elements (2 i, 2 i + 1) */

/* theta_i = base^(-2 i / rot_dim), changed for longer contexts: */
#define AG_ROPE_NONE 0
#define AG_ROPE_LINEAR 1  /* theta_i / factor */
#define AG_ROPE_BASE 2    /* base * factor^(rot_dim / (rot_dim - 2)) in the place of base */
/* theta_i * (g + (1 - g) / factor) with a weight g that is 1 for fast pairs and 0 for slow ones:
 * TURNS: g = clamp((r - low) / (high - low), 0, 1), r = original_len * theta_i / 2 pi (the turns
 *        that pair i makes over the original context);
 * INDEX: g = 1 - clamp((i - i0) / max(i1 - i0, 0.001), 0, 1), with n(r) = rot_dim *
 *        ln(original_len / 2 pi r) / (2 ln base) the index that makes r turns,
 *        i0 = max(floor(n(high)), 0) and i1 = min(ceil(n(low)), rot_dim - 1). */
#define AG_ROPE_TURNS 3
#define AG_ROPE_INDEX 4

typedef struct ag_rope_desc {
  int32_t dtype;       /* AGMM_F16 or AGMM_BF16 */
  int32_t head_dim;    /* 2..1024 */
  int32_t rot_dim;     /* rotated elements, even, 2..min(head_dim, 512) */
  int32_t rot_start;   /* first rotated element */
  int32_t pairing;     /* AG_ROPE_HALF or AG_ROPE_INTERLEAVED */
  int32_t scaling;     /* AG_ROPE_NONE .. AG_ROPE_INDEX */
  double base;         /* > 1 */
  double factor;       /* > 0 (scaling != NONE) */
  double original_len; /* > 0, and low < high, both > 0 (TURNS, INDEX) */
  double low, high;
  double magnitude;    /* factor of the cosines and sines; finite in 32 bits */
  const double* thetas; /* host, rot_dim / 2 angles per position in radians in the place of all of
                           the above, or NULL; read by create only */
} ag_rope_desc;

typedef struct ag_rope_handle ag_rope_handle;

/* Defaults: bf16, head_dim = rot_dim = 128, half pairs, no scaling, base 10000, factor 1,
 * low 1, high 4, magnitude 1. */
void ag_rope_desc_init(ag_rope_desc* desc);

/* The angles per position (radians) that create uses: rot_dim / 2 doubles. Host only. */
int ag_rope_thetas(const ag_rope_desc* desc, double* out);

/* A handle holds the angles, as 64-bit fractions of a turn, on the current device (at most 2 KiB):
 * a position times such a fraction, modulo 2^64, is the phase without a rounding, so angles are as
 * exact at position 2^31 as at 1, and no table of cosines is read. */
int ag_rope_create(const ag_rope_desc* desc, ag_rope_handle** out_handle);
int ag_rope_destroy(ag_rope_handle* h); /* synchronizes the device; NULL-safe */

/* y = R x for `batch` x `tokens` x `heads` heads, or, with gradient = 1, y = R^T x.
 *   x, y: device, 2-byte aligned; element (b, t, h, e) at b * batch + t * token + h * head + e of
 *         the given strides (x's may be 0 or negative). y is x with equal strides (in place; those of
 *         a size of 1 count for nothing), or does not overlap it; y's own elements must not overlap.
 *   positions: device int64, element (b, t) at b * pos_batch + t (pos_batch 0: shared).
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED (over 2^20 heads), WRONG_DEVICE or HIP; zero sizes
 * enqueue nothing. */
int ag_rope_run(ag_rope_handle* h, const void* x, int64_t x_batch, int64_t x_token, int64_t x_head,
                void* y, int64_t y_batch, int64_t y_token, int64_t y_head, const int64_t* positions,
                int64_t pos_batch, int64_t batch, int64_t tokens, int64_t heads, int gradient,
                void* hip_stream);

/* ---- the paged key-value cache ----
 * Pages of page_size rows for each kv head; a row holds one token's head. Slot s is row
 * s % page_size of page s / page_size. Storage of a row:
 *   AG_KV_16BIT: head_dim values of `dtype`;
 *   AG_KV_MXFP8: head_dim e4m3 codes (one byte), and a scale byte for each 32 of them;
 *   AG_KV_MXFP4: head_dim e2m1 codes (element 2 j in the low half of byte j), and the same scales.
 * Scale byte s stands for 2^(s - 127) and is the least, from 1 on, with max |x| <= M 2^(s - 127)
 * over its 32 values (M = 448 for e4m3, 6 for e2m1); codes are x / 2^(s - 127) rounded to nearest,
 * ties to even, and at most the largest code whose value `dtype` can hold. So every code reads
 * back as an exact value of `dtype`. 32 values with a NaN or an infinity among them get scale byte
 * 255 and read back as NaN. A row has its head_dim / 32 scale bytes first and then as many unused
 * ones as fill up 4 bytes. */
#define AG_KV_16BIT 0
#define AG_KV_MXFP8 1
#define AG_KV_MXFP4 2

typedef struct ag_kv_cache {
  int32_t dtype, storage;
  int32_t head_dim;  /* 16BIT: a multiple of 8 up to 256; else a multiple of 32 up to 256 */
  int32_t kv_heads, page_size;
  int32_t reserved;  /* 0 */
  int64_t num_pages; /* num_pages * page_size < 2^31 */
  void *k, *v;       /* device, 16-byte aligned */
  int64_t page_stride, head_stride, row_stride; /* bytes, of k and of v: multiples of 16, >= 0;
                                                   pages and rows below 2^32 apart */
  void *k_scale, *v_scale; /* device, 4-byte aligned; NULL for 16BIT */
  int64_t scale_page, scale_head, scale_row;    /* the same of the scales: multiples of 4 */
} ag_kv_cache;

/* Writes the keys and values of `tokens` tokens to their slots.
 *   k, v: device, 2-byte aligned; element (t, h, e) at t * token + h * head + e. v may be a view
 *         of the same tensor as k.
 *   slots: device int64 [tokens]. A slot < 0 or >= num_pages * page_size: that token is left out.
 *         Two tokens of one call with one slot leave that row undefined (parts of either, and in a
 *         quantised cache one's codes under the other's scales), and no other.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_kv_append(const ag_kv_cache* cache, const void* k, int64_t k_token, int64_t k_head,
                 const void* v, int64_t v_token, int64_t v_head, const int64_t* slots,
                 int64_t tokens, void* hip_stream);

/* The step in front of the attention in one launch: q_out = R q for q_heads heads (as ag_rope_run),
 * and the cache's slots get R k and v (as ag_rope_run into a tensor of `dtype` and then
 * ag_kv_append would leave them, bit for bit). rope must have the cache's dtype and head_dim.
 *   positions: device int64 [tokens]. A token whose slot is left out still has its q rotated.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED, WRONG_DEVICE or HIP. */
int ag_kv_append_rope(const ag_kv_cache* cache, ag_rope_handle* rope, const void* q,
                      int64_t q_token, int64_t q_head, int64_t q_heads, void* q_out,
                      int64_t qo_token, int64_t qo_head, const void* k, int64_t k_token,
                      int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                      const int64_t* positions, const int64_t* slots, int64_t tokens,
                      void* hip_stream);

/* Reads the rows at `slots` back as values of `dtype`: k_out and v_out, element (t, h, e) at
 * t * token + h * head + e, 2-byte aligned. A slot out of range (above) gives zeros.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED or HIP. */
int ag_kv_read(const ag_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out,
               int64_t k_token, int64_t k_head, void* v_out, int64_t v_token, int64_t v_head,
               void* hip_stream);

/* ---- attention of one new token of every sequence ----
 * For sequence b and q head h, with kv head h / (q_heads / kv_heads) and tokens t in
 * [first, len_b), first = max(0, len_b - window) (0 without a window):
 *     s_t = scale * q . k_t, or soft_cap * tanh(scale * q . k_t / soft_cap)
 *     out = sum_t exp(s_t) v_t / sum_t exp(s_t),   lse = ln sum_t exp(s_t)
 * No token to attend to (a length of 0, every page absent): out = 0, lse = -infinity.
 * The sequences' tokens are shared out evenly over the workgroups, or their waves, on the device
 * (lengths are read there), so one long sequence fills the chip as many short ones do; where several
 * share a sequence's head, the last of them to finish joins their partial results in a fixed
 * order. Results do not depend on timing. */
typedef struct ag_attn_desc {
  int32_t dtype, storage;
  int32_t head_dim;          /* as in ag_kv_cache */
  int32_t q_heads, kv_heads; /* q_heads a multiple of kv_heads */
  int32_t num_wgs;           /* workgroups, at most 1024; 0 = auto (fills the chip once) */
  int64_t window;            /* tokens attended to, the new one among them; 0 = all */
  float scale;               /* > 0; 0 = 1 / sqrt(head_dim) */
  float soft_cap;            /* > 0; 0 = none */
} ag_attn_desc;

typedef struct ag_attn_handle ag_attn_handle;

/* Defaults: bf16, 16-bit storage, head_dim 128, 1 q and 1 kv head, the rest 0. */
void ag_attn_desc_init(ag_attn_desc* desc);

/* Device bytes of the workspace (partial results and counters), or a negative code. Host only;
 * sized for 256 compute units. */
int64_t ag_attn_workspace_bytes(const ag_attn_desc* desc);

/* A handle on the current device. workspace as for ag_matmul_create: NULL, or the caller's, 256-byte
 * aligned and of at least ag_attn_workspace_bytes(desc) bytes. Create clears the counters and waits
 * for that; every run leaves them cleared. One run at a time may be in flight for a handle. */
int ag_attn_create(const ag_attn_desc* desc, void* workspace, size_t workspace_bytes,
                   ag_attn_handle** out_handle);
int ag_attn_destroy(ag_attn_handle* h); /* synchronizes the device; NULL-safe */

/* One run.
 *   cache: dtype, storage, head_dim and kv_heads of the handle's desc.
 *   q: device [batch][q_heads][head_dim], element (b, h, e) at b * q_batch + h * q_head + e;
 *   page_table: device int32, entry (b, j) at b * table_row + j, j < table_len: the page of tokens
 *         [j * page_size, (j + 1) * page_size). A page outside [0, num_pages) is absent: its tokens
 *         are left out, and nothing is read there.
 *   lens: device int32 [batch], the new token counted in. < 0 counts as 0; tokens past
 *         table_len * page_size are left out.
 *   out: device, element (b, h, e) at b * o_batch + h * o_head + e, overlapping nothing read;
 *   lse: device float [batch][q_heads], or NULL. q and out 2-byte, the rest 4-byte aligned.
 * Returns AGMM_OK, INVALID_ARG, UNSUPPORTED, WRONG_DEVICE or HIP. */
int ag_attn_run(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                int64_t q_head, const int32_t* page_table, int64_t table_row, int64_t table_len,
                const int32_t* lens, int64_t batch, void* out, int64_t o_batch, int64_t o_head,
                float* lse, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* AGMM_ATTN_H */
