/*
 * gdn_kvcache.h -- C ABI of the serving side of the softmax-attention layers (B200, sm_100a): a
 * paged key/value cache, its tables, and the attention that reads it for a batch of sequences
 * which share a prefix.  Beside gdn_decode.h (the GDN layers' state pool), it is what a serving
 * step of the hybrid model needs for its softmax layers:
 *
 *   gdn_kv_extend      block tables, slots and positions of a step's new tokens, from lengths
 *   gdn_rotary_append  rotary positions on q and k (gdn_rotary.h), k and v into the cache
 *   gdn_prefix_attn    attention of every sequence's L newest tokens over shared prefix + own keys
 *
 * The serving paragraph of "FLARE: Diffusion for Hybrid Language Model" (papernotes.org notes) has two
 * modes; both need the softmax layers at L tokens per sequence: AR-Trust verifies L drafted tokens
 * causally, Diffusion-Trust denoises a block of L tokens that see one another.  L = 1 is plain
 * decoding.
 *
 * Layouts (row-major, contiguous unless strides are given, caller-owned device memory):
 *   k_cache, v_cache [P, p, H_kv, d]   P pages of p tokens, p in {16, 32, 64, 128, 256}
 *   block_table      [N, W] int32      page j of sequence n holds its own tokens [j p, (j+1) p)
 *   prefix_pages     [ceil(Lp / p)] int32  pages of the Lp tokens that every sequence starts with
 *   seq_lens         [N] int32         own tokens of each sequence in the cache (prefix not counted)
 * A slot is page * p + offset.  Device-side integers out of range never lead to an access outside
 * the tensors: they are reported (device_status / the workspace's status word).
 *
 * All calls validate sizes and pointers on the host (no partial launch on error), then enqueue on
 * `stream` and return; nothing is allocated, nothing synchronises, and every call may be captured
 * in a CUDA graph.  Errors: GDN_ERR_INVALID_ARG (sizes, NULL, aliasing), GDN_ERR_ALIGNMENT,
 * GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA (launch failure).
 */
#ifndef GDN_KVCACHE_H
#define GDN_KVCACHE_H

#include "gdn_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- block tables and slot maps
 * num_seqs N >= 1; table_width W >= 1; page_size p >= 1; num_free F >= 0 (entries of free_pages);
 * max_new_tokens M >= 0; prefix_len >= 0 (added to the positions); reserved 0. */
typedef struct {
    int32_t num_seqs;
    int32_t table_width;
    int32_t page_size;
    int32_t num_free;
    int32_t max_new_tokens;
    int32_t prefix_len;
    int32_t reserved[2];
} gdn_kv_extend_desc;

/* Room for new_lens[n] >= 0 more tokens behind the seq_lens[n] >= 0 own tokens of every sequence.
 * The step's tokens are packed by sequence: sequence n has rows [cu_new[n], cu_new[n+1]).  A
 * sequence needs ceil((s+w)/p) - ceil(s/p) new pages, taken in sequence order from the top of the
 * free list: the k-th page taken is free_pages[free_count - 1 - k].
 *   block_table   in/out: the new pages' entries are written, nothing else
 *   seq_lens, new_lens [N], free_pages [F], free_count [1]   int32 (device), read only
 *   slot_map, positions [M]   int32: slot and prefix_len + index of every packed row; rows behind
 *                             the last sequence get -1
 *   cu_new [N+1]; seq_lens_out [N] = s + w; free_left [1] = pages left on the free list
 * Outputs are apart from the inputs, so a call with the same inputs gives the same answer (and
 * writes the same table entries): feed seq_lens_out and free_left to the next step.
 * A sequence is refused (its rows get slot and position -1, its table row stays, its seq_lens_out is
 * its s, it takes no pages) when s or w is negative (w then counts as 0), its tokens s + w would
 * pass W p or INT32_MAX or its rows M, or its pages do not fit: the pages that the sequences up to and with it
 * need (refused ones for the other reasons not counted) pass free_count.  device_status (optional,
 * may be NULL) is cleared, then set to GDN_ERR_INVALID_ARG if any was refused or free_count lies
 * outside [0, F] (it is clamped), or if a row falls on a page id that is negative or whose slot passes
 * INT32_MAX (the row's slot is then -1).  Sums are 64-bit; cu_new and positions saturate at INT32_MAX.
 * Errors: GDN_ERR_INVALID_ARG also when an output overlaps an input or another output. */
gdn_status gdn_kv_extend(const gdn_kv_extend_desc *desc, int32_t *block_table, const int32_t *seq_lens,
                         const int32_t *new_lens, const int32_t *free_pages, const int32_t *free_count,
                         int32_t *slot_map, int32_t *positions, int32_t *cu_new, int32_t *seq_lens_out,
                         int32_t *free_left, int32_t *device_status, gdn_stream_t stream);

/* ---------------------------------------------------------------- rotary + append
 * num_rows R >= 0; num_heads H >= 1; num_kv_heads H_kv >= 1; head_dim d in [1, 256]; rot_dim even,
 * 0 .. d; page_size p and num_pages P >= 1 with p P <= INT32_MAX; strides in elements. */
typedef struct {
    int32_t num_rows;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t rot_dim;
    int32_t interleaved;
    int32_t page_size;
    int32_t num_pages;
    int32_t dtype;
    float scale;
    int64_t q_row_stride, q_head_stride;
    int64_t k_row_stride, k_head_stride;
    int64_t v_row_stride, v_head_stride;
    int64_t q_out_row_stride, q_out_head_stride;
} gdn_append_desc;

/* For every row r with slot s = slot_map[r] >= 0: q_out[r] = rotated q[r], k_cache[s] = rotated k[r],
 * v_cache[s] = v[r].  Rows with slot -1 are padding: nothing of theirs is read or written.  A slot
 * below -1 or not below p P is skipped in the same way and sets device_status (optional; cleared by the
 * call) to GDN_ERR_INVALID_ARG.  Rows that share a slot race: a slot
 * belongs in slot_map once.  The caches have the rows' dtype; gdn_prefix_attn reads bf16 caches.  q_out may be q (same strides); every other overlap of an output (q_out, the
 * caches, device_status) with an input or another output is GDN_ERR_INVALID_ARG, where tensors count as
 * apart as gdn_rotary.h defines it. */
gdn_status gdn_rotary_append(const gdn_append_desc *desc, const uint64_t *turns, const int32_t *positions,
                             const int32_t *slot_map, const void *q, const void *k, const void *v,
                             void *q_out, void *k_cache, void *v_cache, int32_t *device_status,
                             gdn_stream_t stream);

/* ---------------------------------------------------------------- attention with a shared prefix
 * num_seqs N >= 1; num_tokens L >= 1 query tokens per sequence; num_heads H, num_kv_heads H_kv
 * dividing it; head_dim d (64 or 128); page_size p; num_pages P, p P <= INT32_MAX; table_width W >= 0;
 * prefix_len Lp >= 0; causal 0 or 1; dtype GDN_BF16; scale 0 for 1/sqrt(d), else > 0 and
 * finite times log2(e). */
typedef struct {
    int32_t num_seqs;
    int32_t num_tokens;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t page_size;
    int32_t num_pages;
    int32_t table_width;
    int32_t prefix_len;
    int32_t causal;
    int32_t dtype;
    float scale;
} gdn_prefix_attn_desc;

/* Workspace bytes of a call (>= 256, a multiple of 256); 0 when the descriptor is invalid or not
 * supported. */
size_t gdn_prefix_attn_workspace_size(const gdn_prefix_attn_desc *desc);

/* out[n, l, h] = softmax(scale q[n, l, h] . K) V over the Lp prefix keys and the first c own keys of
 * sequence n, key/value head h / (H / H_kv); c = seq_lens[n] when causal = 0 (the L tokens see one
 * another), else max(0, seq_lens[n] - (L - 1 - l)) (token l is the l-th of the L newest).  A row that
 * sees no key is 0; one whose scores are all -inf is NaN, as is one with a score of +inf or NaN.
 *   q, out [N, L, H, d] bf16 (neither out nor the workspace may overlap an input or one another:
 *   GDN_ERR_INVALID_ARG); workspace >= the size above, 256-byte
 *   aligned, contents on entry ignored; its first word is the status that
 *   gdn_dual_read_device_status reads.
 * The prefix is read once for the whole batch, not once per sequence.  What lies in the cache behind
 * a sequence's last token, and every masked key and value, NaN and infinities among them, changes
 * nothing.  Sums and softmax statistics are fp32; probabilities enter the second product as
 * bf16; the output is rounded once.  The same inputs give the same bits on every call.
 * Device-side: seq_lens[n] < 0 or > W p leaves out[n] as it was; a page id outside [0, P) reads as
 * zero keys and values; both set the status to GDN_ERR_INVALID_ARG.  A bounded wait that gives up sets
 * GDN_ERR_TIMEOUT.  Calls that share a workspace and overlap on the GPU race. */
gdn_status gdn_prefix_attn(const gdn_prefix_attn_desc *desc, const void *q, const void *k_cache,
                           const void *v_cache, const int32_t *prefix_pages, const int32_t *block_table,
                           const int32_t *seq_lens, void *out, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream);

/* FOR TESTS of the bounded-wait error path only: gdn_prefix_attn with every device-side wait bounded by
 * `wait_iters` non-blocking polls (>= 1).  A wait that gives up records GDN_ERR_TIMEOUT in the
 * workspace; the kernels then wait with the normal bound for every copy and MMA they issued before
 * they leave; the output is unspecified. */
gdn_status gdn_prefix_attn_test_wait_limit(const gdn_prefix_attn_desc *desc, const void *q, const void *k_cache,
                                           const void *v_cache, const int32_t *prefix_pages,
                                           const int32_t *block_table, const int32_t *seq_lens, void *out,
                                           void *workspace, size_t workspace_bytes, uint32_t wait_iters,
                                           gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_KVCACHE_H */
