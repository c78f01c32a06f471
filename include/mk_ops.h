/*
 * mk_ops — operators on the paged KV pool, outside the fused step (mk.h). On
 * one attention layer: write new rows (rounded or quantised; plain, or with
 * the heads' norm and the position rotation in the same pass), read rows back,
 * and attention of new rows over the cached tokens, the rows a chunk of a text
 * or the nodes of a tree of drafts. On all layers: copy pages, and keep some of
 * a sequence's tokens. And the greedy verification of such a tree. They work on
 * the pool layout and the q8 codec of mk.h, so a context can be installed
 * from dense tensors, saved, moved between an fp16 and a q8 engine, and a
 * prompt chunk can attend to it with any number of rows.
 *
 * Conventions, as in mk.h: sizes are in elements; every call returns an
 * mk_status, checks its arguments before any device work and throws nothing;
 * device code never traps. In addition:
 *  - Every call only queues work on `stream` (a cudaStream_t, NULL = the
 *    legacy default stream) of the current device, allocates nothing and does
 *    not wait, so it can be captured into a CUDA graph. All pointers but the
 *    structs themselves are device pointers of that device.
 *  - The lengths and page tables are read on the device when the work runs. A
 *    page id outside [0, n_pages) names no page: its tokens are unseen by
 *    attention, read as zeros, and a write to them is dropped. row_start is
 *    taken within [0, n_rows], kv_len within [0, 16 * table_stride]; no
 *    value of them makes a kernel leave its buffers.
 */
#ifndef MK_OPS_H_
#define MK_OPS_H_

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MK_OPS_MAX_SEQS 1024

/* Element types of the dense tensors. */
#define MK_F32 0
#define MK_F16 1
#define MK_BF16 2

/* One attention layer of a KV pool (mk_buffers, at that layer's offset):
 * k, v [n_pages][hkv][16][dh] binary16 or int8 codes, and for MK_KV_Q8
 * k_scale, v_scale [n_pages][hkv][16][dh/32] binary16. All 16-byte aligned.
 * dh is a multiple of 64 up to 256. */
typedef struct mk_kv_pool {
    void* k;
    void* v;
    void* k_scale;
    void* v_scale;
    int32_t kv_dtype, n_pages, hkv, dh;
} mk_kv_pool;

/* The rows of a call, in sequence order: rows row_start[s] .. row_start[s+1]-1
 * of the dense tensors are the LAST of sequence s's kv_len[s] tokens (the new
 * rows count among the cached ones), so row r of it is at position
 * kv_len[s] - row_start[s+1] + r. tables[s][i] is the page of its positions
 * 16i .. 16i+15. Rows behind row_start[n_seqs] are left alone. A row at a
 * negative position (more rows than tokens) is dropped by a write, reads as
 * zeros, and sees nothing. Device arrays:
 *   row_start [n_seqs + 1], kv_len [n_seqs], tables [n_seqs][table_stride]
 * n_rows: rows of the dense tensors. max_q: the most rows of one sequence as
 * far as the caller knows (a hint for the choice of a kernel; any value gives
 * the same result up to rounding). */
typedef struct mk_kv_rows {
    const int32_t* row_start;
    const int32_t* kv_len;
    const int32_t* tables;
    int32_t n_seqs, n_rows, table_stride, max_q;
} mk_kv_rows;

/* A dense tensor [rows][heads][dh]: the head dim is contiguous, the other two
 * strides are free (0 and negative ones too, for inputs). */
typedef struct mk_dense {
    void* data;
    int64_t row_stride, head_stride;
} mk_dense;

/*
 * Store rows of K and V ([n_rows][hkv][dh], both of type dtype) at their
 * positions: binary16 round to nearest even, or the q8 codec of mk.h
 * (mk_debug_q8_encode; an infinite value makes its block's scale infinite, so
 * the block reads as NaN; a NaN beside numbers becomes code -127). Two rows of one call must not share a slot (a page
 * that two sequences of the call both write): what it then holds is open.
 * Errors: MK_ERR_INVALID, MK_ERR_UNSUPPORTED (dh), MK_ERR_CUDA.
 */
mk_status mk_kv_write(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_dense* k, const mk_dense* v,
                      int32_t dtype, void* stream);

/*
 * Gather rows of K and V from the pool into dense tensors of type dtype: the
 * stored binary16 value, or scale * code, rounded once to dtype.
 * Errors: as mk_kv_write.
 */
mk_status mk_kv_read(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_dense* k, const mk_dense* v,
                     int32_t dtype, void* stream);

/*
 * Attention of the new rows over the paged cache, which already holds them
 * (mk_kv_write first). Query head h uses kv head h / (hq / hkv). A row at
 * position p sees token t when t <= p, and, with window > 0, when p - t <
 * window or t < sinks. out = sum_t softmax(scale q.k_t) v_t over the seen
 * tokens; a row that sees none (or only scores of -inf) gives 0. With a gate
 * ([n_rows][hq][dh], NULL data for none) the output is multiplied by
 * sigmoid(gate). Values of unseen tokens, infinities and NaN among them, have
 * no effect. Rounding: scores, softmax statistics and sums are fp32; the
 * products' operands are binary16 (bf16 queries are scaled by a power of two
 * per row, exact but for elements below 2^-31 of the row's largest, which are
 * rounded to 2^-39 of it; q8 values and the probabilities are rounded). A q8
 * token with a scale of 512 or more, whose values may pass binary16's largest,
 * enters as 2^-8 of itself: its small values are rounded to 2^-17, the limits of
 * small weights below are 2^8 coarser beside it, and the blocks that meet one
 * take their work twice.
 * q, gate, out: [n_rows][hq][dh] of type dtype (MK_F16 or MK_BF16). out may
 * be q or gate itself; it must not overlap them otherwise.
 * A wait inside the kernel that gives up after two seconds (which takes a
 * fault elsewhere, or lengths that change while it runs) makes the rows it was
 * for NaN; the call's status was returned before. A weight below 2^-36 of the
 * row's largest counts in the sum but adds nothing (an infinite V value that is
 * seen with one gives NaN); from 2^-25 on it has all of binary16's bits.
 * work: mk_attend_work_bytes() bytes, 256-byte aligned, contents free; calls that may
 * overlap on the GPU need a buffer each (two captured graphs too).
 * Errors: MK_ERR_INVALID (also: scale not finite and positive, negative
 * window or sinks, sinks without a window, work too small),
 * MK_ERR_UNSUPPORTED (dh, hq/hkv above 256), MK_ERR_CUDA.
 */
typedef struct mk_attend_args {
    mk_dense q, gate, out;
    int32_t hq, dtype;
    float scale;
    int32_t window, sinks;
    void* work;
    uint64_t work_bytes;
} mk_attend_args;

size_t mk_attend_work_bytes(const mk_kv_pool* pool, const mk_kv_rows* rows, int32_t hq);
mk_status mk_attend(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_attend_args* args, void* stream);

/*
 * Test hook, of the whole process: in the mk_attend calls that follow, waits
 * give up after wait_us (0: the two seconds, the most), and the worker skip_worker (a
 * thread block, or a pair of them; -1: none) never gets its queries, so that its
 * waits run out. Errors: MK_ERR_INVALID.
 */
mk_status mk_debug_attend_wait(int32_t wait_us, int32_t skip_worker);

/*
 * Trees of drafts. The new rows of a sequence may be the nodes of a tree instead
 * of consecutive tokens: parents (device, [n_rows]) holds each row's parent as an
 * index into its sequence's rows. A parent lies before its node; any other value (-1) means
 * that the node follows the cached tokens before the tree, of which there are
 * base = kv_len - rows. Node j lies in slot base + j of the cache, and its position
 * is base + its depth, the number of its ancestors.
 *
 * mk_attend for such rows: node j sees itself, its ancestors and the base tokens;
 * with window > 0 those of them at a position p with pos(j) - p < window or
 * p < sinks. Everything else, errors included, is as mk_attend; parents NULL is
 * mk_attend itself.
 */
mk_status mk_attend_tree(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_attend_args* args, const int32_t* parents,
                         void* stream);

/* Rotation of heads by position (and their norm): dims i and i + rot/2, i < rot/2, of
 * a head turn by position x freq_i; dims from rot on stay. turns (device, [rot/2]):
 * freq_i / 2 pi modulo 1 as 64-bit fractions, from mk_rope_turns. q_gain, k_gain
 * (device, [dh], 16-byte aligned, NULL for none): with a gain, heads of q (k) are
 * first multiplied by (mean of squares + eps)^-1/2 and by it. */
typedef struct mk_rope {
    const uint64_t* turns;
    const float* q_gain;
    const float* k_gain;
    int32_t rot;
    float eps;
} mk_rope;

/* Host only: turns (host, [rot/2]) of freq (host, [rot/2], radians per position), or, when
 * it is NULL, of freq_i = base^(-2i/rot). Errors: MK_ERR_INVALID (rot negative, odd or above
 * 65536, base not positive, a frequency not finite). */
mk_status mk_rope_turns(int32_t rot, double base, const double* freq, uint64_t* turns);

/*
 * New rows of q, k and v, as projected, into use: q normalised and rotated into
 * out, k likewise into the pool, v into the pool (rounded or quantised as by
 * mk_kv_write), in one pass. A row's position for the rotation is positions[row] (device,
 * [n_rows]) or, when that is NULL, by parents, or, when both are, that of its slot.
 * Arithmetic is fp32 (angles: 2^-25 of a turn), each result rounded once.
 * q, out: [n_rows][hq][dh], k, v: [n_rows][hkv][dh], all of type dtype; out may be q
 * itself and must not overlap the inputs otherwise. Rows without a slot have q rotated all
 * the same; rows of no sequence are left alone.
 * Errors: MK_ERR_INVALID (also: parents and positions both given, rot above dh,
 * eps negative), MK_ERR_UNSUPPORTED (dh, rot not a multiple of 64), MK_ERR_CUDA.
 */
typedef struct mk_rope_args {
    mk_dense q, out, k, v;
    int32_t hq, dtype;
    mk_rope rope;
    const int32_t* parents;
    const int32_t* positions;
} mk_rope_args;

mk_status mk_rope_write(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_rope_args* args, void* stream);

/*
 * Greedy verification of trees of drafts. tokens[row] is a node's draft token (a
 * sequence's first row holds the last emitted one, which stands), logits
 * [n_rows][vocab] of type dtype (rows row_stride elements apart) the model's after
 * it. A node's greedy token is the argmax of its logits, the lowest index of
 * several, -1 (which no draft agrees with) when one of them is a NaN. The path
 * starts at the first row and goes on to the lowest child whose token is the
 * greedy token of the node reached. parents NULL: a chain.
 * Outputs (device): per sequence, from row_start on, path [n_rows]: the nodes
 * reached, -1 behind them; emitted [n_rows]: their greedy tokens, i.e. the accepted
 * drafts and one token more, -1 behind them; count [n_seqs]: their number (as
 * mk_step's counts; 0 for a sequence without rows). Rows of no sequence are left alone.
 * work: mk_tree_work_bytes() bytes (0 for few logits), 256-byte aligned, as mk_attend's.
 * Errors: MK_ERR_INVALID, MK_ERR_UNSUPPORTED (vocab or n_rows above 2^30), MK_ERR_CUDA.
 */
typedef struct mk_tree_args {
    const int32_t* parents;
    const int32_t* tokens;
    const void* logits;
    int64_t row_stride;
    int32_t vocab, dtype;
    int32_t* path;
    int32_t* count;
    int32_t* emitted;
    void* work;
    uint64_t work_bytes;
} mk_tree_args;

size_t mk_tree_work_bytes(const mk_kv_rows* rows, int32_t vocab);
mk_status mk_tree_accept(const mk_kv_rows* rows, const mk_tree_args* args, void* stream);

/* Layers of a pool that have their pages in common: pool is the first, and layer i
 * lies i x layer_stride elements of k and v (a 32nd of that of the scales) behind it.
 * layer_stride is a multiple of 256. */
typedef struct mk_kv_layers {
    mk_kv_pool pool;
    int32_t n_layers;
    int64_t layer_stride;
} mk_kv_layers;

/*
 * Copy page src[i] to page dst[i] (device, [n]) in every layer. A pair with an id
 * outside [0, n_pages) is passed over. A page may be copied several times; one that is
 * written must not be another pair's source or target: what it then holds is open.
 * Errors: MK_ERR_INVALID, MK_ERR_UNSUPPORTED (as the pool's; n above 2^30), MK_ERR_CUDA.
 */
mk_status mk_kv_copy(const mk_kv_layers* layers, const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/*
 * Keep some of each sequence's new rows (the path of mk_tree_accept, or, with all of
 * a context's tokens as rows, what is left of it): keep (device, [n_rows]) lists, from
 * row_start on, indices into the sequence's rows, ascending; the first entry that does
 * not ascend or is out of range ends the list. Row keep[i] moves to slot base + i in
 * every layer, in place. kv_len (device, [n_seqs], NULL for none; not rows->kv_len
 * itself) receives base + the entries kept, at least 0. Slots behind that keep what they hold, and
 * pages wholly behind it are the caller's to free. A row whose slot or target has no page
 * does not move. Sequences of one call must not share pages that a row moves to.
 * Errors: MK_ERR_INVALID, MK_ERR_UNSUPPORTED (as the pool's and the rows'; n_rows above
 * 2^30), MK_ERR_CUDA.
 */
mk_status mk_kv_keep(const mk_kv_layers* layers, const mk_kv_rows* rows, const int32_t* keep, int32_t* kv_len, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MK_OPS_H_ */
