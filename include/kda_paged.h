/*
 * kda_paged.h - C ABI of libkda.so for the full-attention layers of a hybrid stack: rotary
 * positions, a paged KV cache, attention of new tokens over it, and the pages' bookkeeping.
 *
 * A hybrid stack alternates KDA layers (kda.h) with full-attention layers, whose sequences hold
 * a KV cache ("Kimi Linear" explainer: three KDA layers, then one full-attention layer).
 *
 * Conventions are those of kda.h: device pointers owned by the caller, work enqueued on
 * `stream`, argument errors reported before anything is enqueued, nothing allocated, no
 * exception across the ABI, contents not checked on the host. The library is entered with the
 * device of the pointers current. In addition:
 *  - Every device index is checked where it is used. A block-table entry outside
 *    [0, num_pages) names no page: its keys are not seen and nothing is stored there. cu_seqlens
 *    values are clamped to [0, total_tokens].
 *  - Calls may be captured into a graph; graphs and calls that share a workspace or change the
 *    same tables must not run at the same time.
 *
 * The cache: k_pages and v_pages are [num_pages][num_kv_heads][page_size][head_dim], elements
 * of dtype; consecutive pages are *_page_stride elements apart (a pool may interleave layers or
 * K and V). page_size is 16, 32, 64, 128 or 256. block_table is int32 [num_seqs][max_pages],
 * rows table_stride elements apart: entry j of row n holds the tokens j * page_size ..
 * (j + 1) * page_size - 1 of sequence n. seq_lens is int32 [num_seqs], each sequence's length.
 * page_refs is int32 [num_pages]: the number of table entries that hold the page; 0 is free.
 * Limits: num_pages <= 2^30, num_seqs <= 2^20, heads <= 4096, total_tokens <= 2^30 (attention:
 * total_tokens * num_q_heads <= 2^30, and keys from 2^31 - 65536 on are not seen).
 *
 * New tokens: sequence n's new tokens are rows cu_seqlens[n] .. cu_seqlens[n + 1] - 1 of
 * q, k, v, o (cu_seqlens NULL: total_tokens / num_seqs rows each, which must divide), and are
 * its LAST tokens: seq_lens counts them, and new token i of m has position seq_lens[n] - m + i.
 * Rows behind the last sequence's are neither read nor written. q, k, v are [rows][heads][dim]
 * with rows *_stride elements apart (a slice of a fused projection is taken as it is).
 *
 * Alignment: every pointer to q, k, v, o and pages 16 bytes, every row and page stride a multiple of
 * 16 bytes, int32 and fp32 arrays 4 bytes, fp64 arrays 8 bytes, workspaces 256 bytes.
 */
#ifndef KDA_PAGED_H_
#define KDA_PAGED_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions ("rotary position embedding": each pair of channels of a head is turned by an
 * angle proportional to the token's position). For pair i < rot_dim / 2 at position p, with
 * a = p * inv_freq[i]:
 *     y1 = scale (x1 cos a - x2 sin a),   y2 = scale (x2 cos a + x1 sin a)
 * The pair is channels (i, i + rot_dim / 2), or (2 i, 2 i + 1) with KDA_ROPE_INTERLEAVED.
 * Channels from rot_dim on are copied. With KDA_ROPE_INVERSE a is negated: that is the
 * gradient, since the transpose of a turn is the turn back (scale is kept).
 * The angle is formed and reduced to one turn in fp64, so positions of any int32 value keep
 * fp32 accuracy; sine, cosine and products are fp32; outputs are rounded once.
 *   q, k      : [num_tokens][num_q_heads | num_k_heads][head_dim] dtype, rows *_stride elements
 *               apart; either may be NULL with its output (then its head count is ignored)
 *   positions : int32 [num_tokens], any value
 *   inv_freq  : fp64 [rot_dim / 2], radians per position
 *   q_out, k_out : q or k itself (in place, with its stride; then q and k may lie between each
 *               other but not overlap), or contiguous and not overlapping q, k or each other
 * head_dim: a multiple of 16 up to 512; rot_dim: a multiple of 16, 16 <= rot_dim <= head_dim.
 */
enum { KDA_ROPE_INTERLEAVED = 1u, KDA_ROPE_INVERSE = 2u };
kda_status kda_rope(const void* q, const void* k, const int32_t* positions, const double* inv_freq,
                    int64_t num_tokens, int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim,
                    int32_t rot_dim, int64_t q_stride, int64_t k_stride, kda_dtype dtype,
                    uint32_t rope_flags, float scale, void* q_out, void* k_out, void* stream);

/*
 * Stores the new tokens' k and v in their sequences' pages, and with inv_freq turns k (before it
 * is stored) and q by their positions on the way: one launch between a layer's projections and
 * its attention. A token whose position is negative or lies in no page is not stored.
 *   q, q_out : as in kda_rope, or both NULL; q_out holds the turned q (with inv_freq NULL q must be
 *              NULL). Either q itself (whose rows then do not overlap those of k and v) or contiguous.
 *   k, v     : [rows][num_kv_heads][head_dim]
 * head_dim: a multiple of 16 up to 512. rope_flags: KDA_ROPE_INTERLEAVED or 0.
 */
kda_status kda_cache_append(const void* q, const void* k, const void* v, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, void* k_pages, void* v_pages,
                            int64_t k_page_stride, int64_t v_page_stride,
                            const int32_t* block_table, int64_t table_stride,
                            const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t num_seqs,
                            int64_t total_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t num_pages, int32_t max_pages,
                            int32_t page_size, kda_dtype dtype, const double* inv_freq,
                            int32_t rot_dim, uint32_t rope_flags, float scale, void* q_out,
                            void* stream);

/*
 * Causal attention of the new tokens over their sequences' pages (which hold the new tokens'
 * k and v already). For the token at position p of sequence n, query head h reading K/V head
 * h / (num_q_heads / num_kv_heads):
 *     s_j = scale q . k_j,   o = sum_j softmax(s)_j v_j,   lse = log sum_j e^{s_j}
 * over the keys j <= p, j > p - window (window 0: all of them) that lie in a page. A row with no
 * key gives o = 0 and lse = -inf, as does a row whose every score is -inf. What lies in unseen
 * places (other pages, the rest of the last page, later tokens, left of the window) does not
 * reach the result, whatever its value.
 *   o   : [rows][num_q_heads][head_dim] dtype, contiguous
 *   lse : fp32 [rows][num_q_heads], or NULL
 * head_dim 64, 128 or 256; num_q_heads a multiple of num_kv_heads; scale positive and finite.
 * Scores, softmax and sums are fp32; with bf16 the weights enter the second product as bf16.
 * Results are the same bit for bit on every run. The workspace depends on the arguments of
 * kda_attn_paged_workspace_size only (0 for arguments the call refuses); its contents need not be initialised.
 */
size_t kda_attn_paged_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t num_q_heads,
                                     int32_t num_kv_heads, int32_t head_dim, kda_dtype dtype);
kda_status kda_attn_paged(const void* q, int64_t q_stride, const void* k_pages,
                          const void* v_pages, int64_t k_page_stride, int64_t v_page_stride,
                          const int32_t* block_table, int64_t table_stride,
                          const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t num_seqs,
                          int64_t total_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t num_pages, int32_t max_pages,
                          int32_t page_size, kda_dtype dtype, float scale, int32_t window, void* o,
                          float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Page bookkeeping. Every choice is by the lowest index, so tables and counts are the same on
 * every run. All arrays are int32 on the device and are changed in place.
 */

/* A pool of pages (or of any per-slot data: KDA states too): `outer` planes (layers, K and V)
 * outer_stride bytes apart, each of num_pages pages of page_bytes bytes, page_stride bytes apart.
 * base 16-byte aligned, the other sizes multiples of 16 bytes. Pages may not overlap. */
typedef struct {
  void* base;
  int64_t outer_stride, page_stride, page_bytes;
  int32_t outer, num_pages;
} kda_page_pool;
enum { KDA_MAX_POOLS = 8 };

/*
 * Room for more tokens: request i adds new_tokens[i] tokens to sequence seqs[i] (seqs NULL:
 * sequence i, count = num_seqs). Each takes the lowest free pages, in the order of the requests;
 * its table row gets them, page_refs becomes 1, seq_lens grows. granted[i] is 1, or 0 where
 * nothing was done: no such sequence, a sequence that an earlier request names, a negative
 * count or length, a row that is too short, or too few free pages for it and the well-formed requests
 * before it (one that needs no page is granted). A sequence's last page has to be its own
 * (kda_pages_fork leaves it so).
 */
size_t kda_pages_plan_workspace_size(int32_t count, int32_t num_seqs, int32_t num_pages);
kda_status kda_pages_alloc(int32_t* page_refs, int32_t* block_table, int64_t table_stride,
                           int32_t* seq_lens, const int32_t* seqs, const int32_t* new_tokens,
                           int32_t count, int32_t num_seqs, int32_t num_pages, int32_t max_pages,
                           int32_t page_size, int32_t* granted, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Fork: sequence children[i] becomes a copy of sequence parents[i]. They share the full pages
 * (page_refs grows); a page that is not full is copied, in every pool, to the lowest free page.
 * granted[i] is 1, or 0 where nothing was done: no such parent or child, a child that is not
 * empty before the call or that an earlier pair names, a length outside the row, or too few
 * free pages for it and the well-formed pairs before it. A parent may be named often. num_pools 0: the bookkeeping
 * alone.
 */
kda_status kda_pages_fork(const kda_page_pool* pools, int32_t num_pools, int32_t* page_refs,
                          int32_t* block_table, int64_t table_stride, int32_t* seq_lens,
                          const int32_t* parents, const int32_t* children, int32_t count,
                          int32_t num_seqs, int32_t num_pages, int32_t max_pages,
                          int32_t page_size, int32_t* granted, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Free: the sequences seqs[i] become empty. Each entry that they hold leaves page_refs one
 * lower and becomes -1; seq_lens becomes 0. No such sequence, an empty one, or one named twice: nothing
 * more is done.
 */
kda_status kda_pages_free(int32_t* page_refs, int32_t* block_table, int64_t table_stride,
                          int32_t* seq_lens, const int32_t* seqs, int32_t count, int32_t num_seqs,
                          int32_t num_pages, int32_t max_pages, int32_t page_size, void* stream);

/*
 * Compaction: while a live page (page_refs > 0) lies above a free one, the highest live page
 * moves to the lowest free page, in every pool; afterwards the live pages are 0 .. live - 1.
 * out_refs and out_table get the new counts and table (every entry that names a moved page is
 * rewritten, whatever the lengths); they may be page_refs and block_table themselves. moved[0] is
 * the number of pages moved.
 */
size_t kda_pages_compact_workspace_size(int32_t num_pages);
kda_status kda_pages_compact(const kda_page_pool* pools, int32_t num_pools,
                             const int32_t* page_refs, const int32_t* block_table,
                             int64_t table_stride, int32_t num_seqs, int32_t num_pages,
                             int32_t max_pages, int32_t* out_refs, int32_t* out_table,
                             int64_t out_table_stride, int32_t* moved, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Copies page src[i] to page dst[i] in every pool, i < count. Pairs with an index outside the
 * pool, or with src[i] = dst[i], are passed over. No page may be a dst twice, or a dst of one
 * pair and the src of another: the copies run in no order.
 */
kda_status kda_pages_copy(const kda_page_pool* pools, int32_t num_pools, const int32_t* src,
                          const int32_t* dst, int32_t count, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_PAGED_H_ */
