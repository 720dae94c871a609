/*
 * si_kv.h -- C ABI of libsimoe, attention block: a paged key/value cache held
 * in 8 bits with one scale for each page (block of tokens) and head, the
 * attention that reads it, and the eviction that keeps it within a budget.
 * It is the other half of a decoder layer whose FFN si_moe.h runs; the
 * conventions (ownership, streams, alignment, errors, threading) are that
 * header's.  Every call is stream-ordered, allocates nothing, never
 * synchronises (except si_kv_read_status) and can be captured in a CUDA graph.
 *
 * The cache.  A sequence's tokens lie in pages of P tokens (16, 32 or 64).
 * Page p of K holds, for each of the Hkv kv heads, P rows of D codes
 * (k_codes [n_pages][Hkv][P][D], row = token) and one fp32 scale
 * (k_scale [n_pages][Hkv]); V likewise.  A value is code * scale.  Codes are
 * int8 (-127..127) or FP8 E4M3.
 * A page is quantised once, when its last token arrives, from the 16-bit
 * values; its codes do not depend on how the tokens came in.  Until then the
 * tokens are held in 16 bits in a ring of 2P rows for each sequence slot
 * (k_tail [n_slots][Hkv][2P][D]): token t in row t mod 2P.  The ring also
 * keeps the new tokens of the page before, so a step of at most P tokens can
 * be taken back, whole or in part, by using a smaller length afterwards.
 * Quantisation of a page and head: amax = max|x| over its P*D values;
 * scale = fp32(amax / Q), code = round-half-even(x * fp32(Q / amax)) with
 * Q = 127 (int8), or the nearest E4M3 value with Q = 448.  amax < 2^-100:
 * scale 0, codes 0.  A page with a non-finite value gets the scale NaN and
 * zero codes, so that whatever attends to a token of that page is NaN.
 *
 * A call's sequences (si_kv_batch).  Sequence b has lens[b] tokens in the
 * cache and n_b = q_start[b+1] - q_start[b] rows in q, k and v.  Row i of
 * sequence b is row q_start[b] + i.  page_table[b][j] is the page that holds
 * tokens jP .. jP+P-1.  These arrays are in device memory; the host gives
 * bounds on what they hold (max_new, max_len, total_new).  A sequence whose
 * entries break a bound is treated as having no rows (and no tokens), and a
 * page or slot index outside the cache is not followed (what would attend to
 * it is NaN; what would be written there is not): both set SI_ERR_DEVICE,
 * which si_kv_read_status returns.
 */
#ifndef SI_KV_H
#define SI_KV_H

#include "si_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SI_KV_INT8 1              /* si_kv_desc.code */
#define SI_KV_E4M3 2
#define SI_KV_BF16 1              /* si_kv_desc.dtype */
#define SI_KV_F16 2
#define SI_KV_MAX_SEQS 1024       /* sequences of one call */
#define SI_KV_MAX_HEADS 256       /* query heads */
#define SI_KV_MAX_LEN (1 << 22)   /* tokens of one sequence */
#define SI_KV_MAX_EVICT_PAGES 16384 /* pages of one sequence in si_kv_evict */

/* n_heads is a multiple of n_kv_heads (query head h reads kv head
 * h / (n_heads / n_kv_heads)); head_dim 64, 128 or 256; page_tokens 16, 32 or
 * 64; code SI_KV_INT8 or SI_KV_E4M3; dtype the 16-bit type of q, k, v, out and
 * the ring, SI_KV_BF16 or SI_KV_F16. */
typedef struct si_kv_desc {
    int32_t n_heads;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t page_tokens;
    int32_t code;
    int32_t dtype;
} si_kv_desc;

typedef struct si_kv_plan_s *si_kv_plan_t;

/* The cache's buffers (device pointers, 16-byte aligned; owned by the caller). */
typedef struct si_kv_cache {
    void *k_codes;      /* [n_pages][Hkv][P][D] 8-bit codes */
    void *v_codes;
    float *k_scale;     /* [n_pages][Hkv] */
    float *v_scale;
    void *k_tail;       /* [n_slots][Hkv][2P][D] 16-bit ring */
    void *v_tail;
    int64_t n_pages;
    int32_t n_slots;
} si_kv_cache;

typedef struct si_kv_batch {
    int32_t n_seqs;             /* 1..SI_KV_MAX_SEQS */
    int32_t total_new;          /* rows of q, k, v, out (>= q_start[n_seqs]) */
    int32_t max_new;            /* no sequence has more rows (nor 2^30 rows times query heads of a kv head) */
    int32_t max_len;            /* no sequence has more tokens, the call's new ones counted */
    const int32_t *q_start;     /* [n_seqs + 1] first row of each sequence, ascending */
    const int32_t *lens;        /* [n_seqs] tokens in the cache (si_kv_append: before the call) */
    const int32_t *page_table;  /* [n_seqs][table_stride] page indices */
    const int32_t *slots;       /* [n_seqs] ring slot of each sequence, all different; NULL: sequence b has slot b */
    int32_t table_stride;       /* >= max_len / page_tokens */
} si_kv_batch;

/* A 16-bit [rows][heads][D] operand: element (r, h, d) is at r*row_stride +
 * h*head_stride + d (strides in elements, multiples of 8), so the three parts
 * of a fused projection need no copy.  data (and si_kv_weigh's lse) may be NULL
 * where total_new is 0. */
typedef struct si_kv_rows {
    void *data;
    int64_t row_stride;
    int64_t head_stride;
} si_kv_rows;

/* Validate desc and choose launch shapes for device cuda_device.  Host memory
 * only.  *out receives a plan to free with si_kv_plan_destroy. */
si_status si_kv_plan(const si_kv_desc *desc, int cuda_device, si_kv_plan_t *out);
void si_kv_plan_destroy(si_kv_plan_t plan);

/* Bytes of device scratch that the calls with these batch bounds need (one
 * size for all of them; a buffer for larger bounds serves smaller ones). */
si_status si_kv_scratch_bytes(si_kv_plan_t plan, int32_t n_seqs, int32_t total_new, int32_t max_new,
                              int32_t max_len, size_t *bytes);
/* Zero the scratch control block, stream-ordered.  Once, before the first call. */
si_status si_kv_scratch_init(si_kv_plan_t plan, void *scratch, size_t scratch_bytes, si_stream_t stream);

/* Append the rows of k and v to the cache: lens[b] tokens become
 * lens_out[b] = lens[b] + n_b.  Pages whose last token arrives are quantised
 * (their page_table entries must name free pages; the unfinished page needs
 * none yet); the new rows of the unfinished page and of the one before it go
 * into the ring.  lens_out [n_seqs] must not overlap lens. */
si_status si_kv_append(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *k,
                       const si_kv_rows *v, int32_t *lens_out, void *scratch, size_t scratch_bytes,
                       si_stream_t stream);

/* Read n pages back: k_out, v_out [n][Hkv][P][D] in the plan's 16-bit type,
 * the nearest value to fp32(code * scale).  pages [n]: device page indices. */
si_status si_kv_read(si_kv_plan_t plan, const si_kv_cache *cache, const int32_t *pages, int32_t n, void *k_out,
                     void *v_out, void *scratch, size_t scratch_bytes, si_stream_t stream);

/* Causal attention of each sequence's last n_b tokens (lens counts them; they
 * have been appended): row i sees tokens 0 .. lens[b] - n_b + i.
 * (The kernel goes by max_new: a chunk of a prompt and the steps of many other
 * sequences are faster in two calls than in one.)
 * out[row][h] = sum_t softmax_t(sm_scale * q[row][h] . k_t) v_t, and, where lse
 * is not NULL, lse[row][h] = log sum_t exp(sm_scale * q . k_t) ([total_new]
 * [n_heads] fp32).  A row that sees no token (lens[b] < n_b) gives zeros and
 * lse -inf.  Scores are held in 32 bits: one below their range has no weight, and
 * a row with one above it, or with all of its scores below it, is NaN.  out
 * must not overlap q (checked where their strides are the same), and its rows and
 * heads must not overlap one another. */
si_status si_kv_attend(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *q,
                       const si_kv_rows *out, float *lse, float sm_scale, void *scratch, size_t scratch_bytes,
                       si_stream_t stream);

/* Add the attention weights that the rows of q gave each cached token to its
 * running sum: acc_out[b][g][t] = decay * acc_in[b][g][t] + sum over the n_b rows
 * and the query heads of kv head g of exp(sm_scale * q . k_t - lse[row][h]),
 * for t < lens[b]; entries past that are not written.  The call's own tokens
 * (the last n_b) have no earlier sum: acc_in is read for t < lens[b] - n_b
 * only, and may be NULL (no earlier sums at all).  q and lse are those of
 * si_kv_attend, or of a prompt's last rows alone: then the prompt's tokens before
 * those rows count as old, and the caller zeroes their entries of acc_in first
 * (si_kv_evict leaves old sums past its new lengths).  acc_in, acc_out:
 * [n_seqs][Hkv][acc_stride] fp32, acc_stride >= max_len; they may be the same
 * array.  The sums are taken in a fixed order (the same inputs give the same
 * bits). */
si_status si_kv_weigh(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *q,
                      const float *lse, const float *acc_in, float *acc_out, int64_t acc_stride, float decay,
                      float sm_scale, void *scratch, size_t scratch_bytes, si_stream_t stream);

/* Evict by accumulated weight: each kv head of each sequence keeps at most
 * `budget` of its F = lens[b] / P full pages (and the unfinished page): the
 * first `sink`, the last `recent`, and of the others those with the largest sum
 * of acc over their tokens (exact to 2^-49 of a page's largest value, in any order of
 * its tokens; ties stay with the lower page; NaN counts as largest), in their order.  The kept pages' codes and scales
 * are copied as they are to the pages new_table[b][0 .. min(F, budget) - 1],
 * so they are not rounded again; which page a slot of the new table holds may
 * differ from head to head.  new_table names pages that no sequence of the
 * call uses.  acc_out gets the kept tokens' sums (entries past the new length
 * are not written); keep[b][g][i] the kept page numbers, -1 past their count;
 * lens_out[b] = min(F, budget) * P + lens[b] mod P.  The unfinished page's rows
 * go to the ring place of the new length in slot new_slots[b] (NULL: the
 * batch's own slots): the sequence's own slot, or one that holds no unfinished
 * rows of another sequence of the call and is not another's new one (else
 * SI_ERR_DEVICE, and the rows stay where they are).  The rows of the page before are
 * not carried over: a step cannot be taken back past an eviction's page
 * boundary.  The old pages are left as they are.  sink + recent <=
 * budget; max_len / P <= SI_KV_MAX_EVICT_PAGES; acc_stride >= max_len for both;
 * acc_out and lens_out must not overlap acc_in and lens; q_start is not read. */
si_status si_kv_evict(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const float *acc_in,
                      float *acc_out, int64_t acc_stride, int32_t budget, int32_t sink, int32_t recent,
                      const int32_t *new_table, const int32_t *new_slots, int32_t *keep, int32_t *lens_out,
                      void *scratch, size_t scratch_bytes, si_stream_t stream);

/* Synchronise `stream`, return the device status recorded in `scratch` since
 * the last read (SI_OK if none) and clear it. */
si_status si_kv_read_status(si_kv_plan_t plan, const void *scratch, si_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SI_KV_H */
