/*
 * mk_ops — operators on one attention layer of the paged KV pool, outside the
 * fused step (mk.h): write new rows (rounded or quantised), read rows back,
 * and attention of a chunk of new rows over the cached tokens. They work on
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

#ifdef __cplusplus
}
#endif
#endif /* MK_OPS_H_ */
