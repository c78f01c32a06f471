// Moves of cached tokens within the pool, in all layers of one call: whole pages
// (a prefix for another sequence) and kept tokens (the accepted path of a tree of
// drafts, or a context that loses old tokens). Nothing is computed: both are bound by
// HBM traffic when much moves, by the launch when little does. Measured: 3 x 256 pages in 17
// layers copied in 168 us (binary16, 1.14 GB, 6.8 TB/s, the copy rate) and 92 us (q8, 606 MB,
// 6.6 TB/s); 8,176 of 23,000 tokens moved in 17 layers (q8, 605 MB) in 128 us, 4.7 TB/s (a column's
// batches follow each other: the latency of 64 of them); the paths of four trees in 17 layers in 5 us.
#include <cuda_runtime.h>

#include "ops_internal.cuh"

namespace mk {
namespace ops {
namespace {

// -------------------------------------------------------------------- pages
// K and V of a page are contiguous, [kv heads][16][dh], and so are their scales: a
// block copies one chunk of one of them, in one layer.
constexpr int kCopyBlock = 256;

struct CopyArgs {
  mk_kv_layers l;
  const int32_t* src;
  const int32_t* dst;
  int n, chunks, scale_chunks;  // pairs of pages; chunks of a page's K (V), of its scales
  int64_t page_bytes, scale_bytes;
};

template <int U>
__global__ void __launch_bounds__(kCopyBlock) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
  wait_for_previous();
  const int64_t layer = static_cast<int64_t>(blockIdx.z) * a.l.layer_stride;
  const bool q8 = a.l.pool.kv_dtype == MK_KV_Q8;
  int chunk = blockIdx.x;
  const bool scales = chunk >= 2 * a.chunks;
  if (scales) chunk -= 2 * a.chunks;
  const int per = scales ? a.scale_chunks : a.chunks;
  const bool v = chunk >= per;
  if (v) chunk -= per;
  const int64_t bytes = scales ? a.scale_bytes : a.page_bytes;
  uint8_t* const base = static_cast<uint8_t*>(scales ? (v ? a.l.pool.v_scale : a.l.pool.k_scale) : v ? a.l.pool.v : a.l.pool.k) +
                        (scales ? layer / 16 : q8 ? layer : 2 * layer);
  const int64_t at = static_cast<int64_t>(chunk) * (kCopyBlock * 16 * U) + threadIdx.x * 16;
  for (int pair = blockIdx.y; pair < a.n; pair += gridDim.y) {
    const int s = a.src[pair], d = a.dst[pair];
    if (s < 0 || s >= a.l.pool.n_pages || d < 0 || d >= a.l.pool.n_pages) continue;
    const uint8_t* from = base + s * bytes;
    uint8_t* to = base + d * bytes;
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at + u * kCopyBlock * 16 < bytes) x[u] = *reinterpret_cast<const uint4*>(from + at + u * kCopyBlock * 16);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at + u * kCopyBlock * 16 < bytes) *reinterpret_cast<uint4*>(to + at + u * kCopyBlock * 16) = x[u];
  }
}

// --------------------------------------------------------------- kept tokens
// Entry i of a sequence's list moves new row keep[i] to slot base + i. The list
// ascends, so keep[i] >= i: a slot is written by an entry at or before every entry that
// reads it or a later slot. A block takes one column of a head's rows, or its scales,
// through the whole list, a batch of entries at a time: all of a batch are read, the
// block meets, all are written. What later entries read lies behind everything that
// earlier ones write, so columns need no order among blocks, and the next batch is read
// while this one is on its way: its pages were looked up a batch before, its list's entries
// read two before. LANES lanes of 16 bytes take a token: 4 in long lists (128 entries a
// batch, narrow columns, many blocks), 16 in shorter ones (32 entries).
constexpr int kThreads = 128, kDeep = 4;  // threads of a block, tokens that a thread moves at a time

struct KeepArgs {
  mk_kv_layers l;
  mk_kv_rows rows;
  const int32_t* keep;
  int32_t* kv_len;
  int row_bytes, pieces, data;  // bytes of a head's row, columns of it; columns of a layer that are K's and V's
};

// (Eight blocks an SM: without the limit the narrow one took 56 registers and spilled, 138 against 135 us; looked up behind
// the loads of the next batch, 149 against 128.)
template <int LANES>
__global__ void __launch_bounds__(kThreads, 8) kv_keep_kernel(const __grid_constant__ KeepArgs a) {
  constexpr int kTokens = kThreads * kDeep / LANES;  // entries of a batch
  static_assert(kTokens <= kThreads && kTokens % 32 == 0, "a thread looks at one entry");
  __shared__ int from[3][kTokens], to[3][kTokens];
  __shared__ uint32_t ascends[3][kTokens / 32];
  wait_for_previous();
  const int s = blockIdx.y, tid = threadIdx.x;
  const SeqView v = seq_view(a.rows, s);
  const int base = v.kv_len - v.q_len, hkv = a.l.pool.hkv, n_pages = a.l.pool.n_pages;
  const int64_t layer = static_cast<int64_t>(blockIdx.z) * a.l.layer_stride;
  // the column: its head's first row, the bytes from row to row, and those of a row that it moves
  const int c = blockIdx.x, words = a.l.pool.dh / 64;
  const bool scales = c >= a.data;
  const int col = scales ? c - a.data : c, per = scales ? 1 : a.pieces, kvh = col / per, piece = col - kvh * per;
  const bool is_v = kvh >= hkv;
  const int head = is_v ? kvh - hkv : kvh, bytes = scales ? 4 * words : a.row_bytes;
  uint8_t* p = static_cast<uint8_t*>(scales ? (is_v ? a.l.pool.v_scale : a.l.pool.k_scale) : is_v ? a.l.pool.v : a.l.pool.k) +
               (scales ? layer / 16 : a.l.pool.kv_dtype == MK_KV_Q8 ? layer : 2 * layer) + static_cast<int64_t>(head) * kPage * bytes;
  const int at16 = (piece * LANES + tid % LANES) * 16;
  const bool mine = scales || at16 < bytes;
  if (!scales) p += at16;

  struct Entry {
    int k, before;
  };
  // a thread's entry of batch b of the list, and the one before it
  auto entry = [&](int b) {
    const int i = b * kTokens + tid;
    return tid < kTokens && i < v.q_len ? Entry{a.keep[v.r0 + i], i ? a.keep[v.r0 + i - 1] : -1} : Entry{-1, -1};
  };
  // Batch b, whose entries are e: rows of a head that they come from and go to (-1: does not move), and which entries follow
  // the one before.
  auto look = [&](int b, int buf, Entry e) {
    if (tid >= kTokens) return;
    const int i = b * kTokens + tid;
    int f = -1, t = -1;
    const bool good = e.k < v.q_len && e.k > max(e.before, -1);
    if (good && e.k != i) {
      f = token_at(a.rows, n_pages, s, base + e.k);
      t = token_at(a.rows, n_pages, s, base + i);
      if (f < 0 || t < 0) f = -1;
    }
    from[buf][tid] = f < 0 ? -1 : f / kPage * (hkv * kPage) + f % kPage;  // (below 2^31: check_pool)
    to[buf][tid] = t < 0 ? -1 : t / kPage * (hkv * kPage) + t % kPage;
    const uint32_t ok = __ballot_sync(0xffffffffu, good);
    if (tid % 32 == 0) ascends[buf][tid / 32] = ok;
  };
  struct Batch {
    uint4 x[kDeep];
    int d[kDeep];
    int n;  // entries that count, up to the first that does not follow
  };
  auto load = [&](int buf) {
    Batch t;
    t.n = 0;
#pragma unroll
    for (int w = 0; w < kTokens / 32; ++w) {
      const uint32_t end = ~ascends[buf][w];
      if (t.n == 32 * w) t.n += end ? __ffs(end) - 1 : 32;
    }
    if (scales) {  // a thread a token, its scales word by word
      const int r = tid < t.n ? from[buf][tid] : -1;
      t.d[0] = r < 0 ? -1 : to[buf][tid];
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p + static_cast<int64_t>(r) * bytes);
      if (r >= 0) {
        t.x[0].x = q[0];
        if (words > 1) t.x[0].y = q[1];
        if (words > 2) t.x[0].z = q[2];
        if (words > 3) t.x[0].w = q[3];
      }
    } else {
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int e = u * (kThreads / LANES) + tid / LANES, r = mine && e < t.n ? from[buf][e] : -1;
        t.d[u] = r < 0 ? -1 : to[buf][e];
        if (r >= 0) t.x[u] = *reinterpret_cast<const uint4*>(p + static_cast<int64_t>(r) * bytes);
      }
    }
    return t;
  };
  auto store = [&](const Batch& t) {
    if (scales) {
      if (t.d[0] < 0) return;
      uint32_t* q = reinterpret_cast<uint32_t*>(p + static_cast<int64_t>(t.d[0]) * bytes);
      q[0] = t.x[0].x;
      if (words > 1) q[1] = t.x[0].y;
      if (words > 2) q[2] = t.x[0].z;
      if (words > 3) q[3] = t.x[0].w;
    } else {
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (t.d[u] >= 0) *reinterpret_cast<uint4*>(p + static_cast<int64_t>(t.d[u]) * bytes) = t.x[u];
    }
  };
  look(0, 0, entry(0));
  look(1, 1, entry(1));
  Entry ahead = entry(2);
  __syncthreads();
  Batch now = load(0);
  int count = now.n;
  for (int b = 0, buf = 0;; ++b) {
    // batch b is on its way (or here), the list of batch b + 1 in shared memory
    const int next = buf == 2 ? 0 : buf + 1, after = next == 2 ? 0 : next + 1;
    const bool more = now.n == kTokens;
    Batch then;
    then.n = 0;
    if (more) {
      look(b + 2, after, ahead);  // (its buffer was read two batches ago)
      then = load(next);
      ahead = entry(b + 3);
    }
    __syncthreads();  // every thread has read batch b
    store(now);
    if (!more) break;
    now = then;
    count += now.n;
    buf = next;
  }
  if (a.kv_len && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) a.kv_len[s] = max(base + count, 0);
}

mk_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_kv_copy(const mk_kv_layers* layers, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  using namespace mk::ops;
  const mk_status st = check_layers(layers);
  if (st != MK_OK) return st;
  if (n < 0) return MK_ERR_INVALID;
  if (n > kMaxList) return MK_ERR_UNSUPPORTED;
  if (n == 0) return MK_OK;
  if (!src || !dst) return MK_ERR_INVALID;
  const mk_kv_pool& p = layers->pool;
  const bool q8 = p.kv_dtype == MK_KV_Q8;
  CopyArgs a{*layers, src, dst, n, 0, 0, static_cast<int64_t>(p.hkv) * kPage * p.dh * (q8 ? 1 : 2), static_cast<int64_t>(p.hkv) * p.dh};
  // 16 KB a block, or 4 KB where that leaves SMs without a block (64 KB a pair of pages: 8 pairs 1.6 against 1.4 us, 32
  // pairs 1.7 both, 76 pairs 2.0 against 2.5, 1,000 pairs 21 against 26)
  const bool big = a.page_bytes * 2 * n * layers->n_layers >= (152ll << 14);
  const int64_t span = kCopyBlock * 16 * (big ? 4 : 1);
  const int64_t chunks = (a.page_bytes + span - 1) / span, scale_chunks = q8 ? (a.scale_bytes + span - 1) / span : 0;
  if (2 * (chunks + scale_chunks) > 0x7fffffffll) return MK_ERR_UNSUPPORTED;
  a.chunks = static_cast<int>(chunks);
  a.scale_chunks = static_cast<int>(scale_chunks);
  const dim3 grid(static_cast<unsigned>(2 * (chunks + scale_chunks)), n < 65535 ? n : 65535, layers->n_layers);
  return launched(launch_early(big ? kv_copy_kernel<4> : kv_copy_kernel<1>, grid, dim3(kCopyBlock), 0, static_cast<cudaStream_t>(stream), a));
}

extern "C" mk_status mk_kv_keep(const mk_kv_layers* layers, const mk_kv_rows* rows, const int32_t* keep, int32_t* kv_len, void* stream) {
  using namespace mk::ops;
  mk_status st = check_layers(layers);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (rows->n_rows > kMaxList) return MK_ERR_UNSUPPORTED;
  if (rows->n_seqs == 0) return MK_OK;
  if (!keep && rows->n_rows > 0) return MK_ERR_INVALID;
  const mk_kv_pool& p = layers->pool;
  const bool q8 = p.kv_dtype == MK_KV_Q8;
  // Short lists (drafts) in wide columns, long ones in narrow: the more blocks the more is on its way. (Half of four
  // sequences' rows kept in 17 layers: 16 rows 2.6 against 6.6 us, 128 rows 7.1 against 10, 512 rows 26 against 28; 8,192 of
  // 23,000 tokens 145 in columns twice as wide and 166 in whole rows against 132.)
  const bool wide = rows->n_rows <= 512ll * rows->n_seqs;
  const int width = 16 * (wide ? 16 : 4);
  KeepArgs a{*layers, *rows, keep, kv_len, p.dh * (q8 ? 1 : 2), 0, 0};
  a.pieces = (a.row_bytes + width - 1) / width;
  const int64_t data = 2ll * p.hkv * a.pieces, columns = data + (q8 ? 2ll * p.hkv : 0);
  if (columns > (1 << 24)) return MK_ERR_UNSUPPORTED;
  a.data = static_cast<int>(data);
  const dim3 grid(static_cast<unsigned>(columns), rows->n_seqs, layers->n_layers);
  return launched(launch_early(wide ? kv_keep_kernel<16> : kv_keep_kernel<4>, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a));
}
