// Moves of cached tokens within the pool, in all layers of one call: whole pages
// (a prefix for another sequence) and kept tokens (the accepted path of a tree of
// drafts, or a context that loses old tokens). Nothing is computed: both are bound by
// HBM traffic when much moves, by the launch when little does.
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
    const int s = __ldg(a.src + pair), d = __ldg(a.dst + pair);
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
// reads it or a later slot. A block takes a 64-byte column of a head's rows (or its
// scales) through the whole list, kTokens entries at a time: all are read, the block
// meets, all are written. What later entries read lies behind everything that earlier
// ones write, so columns need no order among blocks, and the next read may begin before
// the write. `per` columns share one look at the list.
constexpr int kTokens = 128;  // threads of a block, and entries at a time
constexpr int kWide = 64;     // bytes of a column

struct KeepArgs {
  mk_kv_layers l;
  mk_kv_rows rows;
  const int32_t* keep;
  int32_t* kv_len;
  int row_bytes, columns, data, per;  // bytes of a head's row; columns of a layer, those of K and V among them; columns of a block
};

__global__ void __launch_bounds__(kTokens) kv_keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int from[kTokens], to[kTokens], first;
  const int s = blockIdx.y, tid = threadIdx.x;
  const SeqView v = seq_view(a.rows, s);
  const int base = v.kv_len - v.q_len, hkv = a.l.pool.hkv, n_pages = a.l.pool.n_pages;
  const int64_t layer = static_cast<int64_t>(blockIdx.z) * a.l.layer_stride;
  const bool q8 = a.l.pool.kv_dtype == MK_KV_Q8;
  const int c0 = blockIdx.x * a.per, c1 = min(c0 + a.per, a.columns);
  int count = 0;
  for (int i0 = 0; i0 < v.q_len; i0 += kTokens) {
    const int i = i0 + tid;
    int f = -1, t = -1;
    bool good = false;
    if (i < v.q_len) {
      const int k = __ldg(a.keep + v.r0 + i), before = i ? __ldg(a.keep + v.r0 + i - 1) : -1;
      good = k < v.q_len && k > max(before, -1);
      if (good && k != i) {
        f = token_at(a.rows, n_pages, s, base + k);
        t = token_at(a.rows, n_pages, s, base + i);
      }
    }
    if (tid == 0) first = kTokens;
    __syncthreads();  // (also: the entries before have been taken from `from` and `to`)
    from[tid] = t < 0 ? -1 : f;
    to[tid] = t;
    if (!good) atomicMin(&first, tid);
    __syncthreads();
    const int n = first;  // entries up to the first that does not ascend
    count += n;
    for (int c = c0; c < c1; ++c) {
      const bool scales = c >= a.data;
      const int per_row = scales ? 1 : a.row_bytes / kWide;
      const int col = scales ? c - a.data : c, piece = col % per_row, kvh = col / per_row, head = kvh % hkv;
      const bool is_v = kvh >= hkv;
      // byte of token row r (page r / 16, slot r % 16) of the column
      auto at = [&](int r, int bytes) { return ((static_cast<int64_t>(r / kPage) * hkv + head) * kPage + r % kPage) * bytes; };
      if (!scales) {
        uint8_t* const p = static_cast<uint8_t*>(is_v ? a.l.pool.v : a.l.pool.k) + (q8 ? layer : 2 * layer) + piece * kWide + tid % 4 * 16;
        uint4 x[4];
        int d[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = u * (kTokens / 4) + tid / 4, r = e < n ? from[e] : -1;
          d[u] = r < 0 ? -1 : to[e];
          if (r >= 0) x[u] = *reinterpret_cast<const uint4*>(p + at(r, a.row_bytes));
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (d[u] >= 0) *reinterpret_cast<uint4*>(p + at(d[u], a.row_bytes)) = x[u];
      } else {
        uint8_t* const p = static_cast<uint8_t*>(is_v ? a.l.pool.v_scale : a.l.pool.k_scale) + layer / 16;
        const int words = a.l.pool.dh / 64, r = tid < n ? from[tid] : -1, d = r < 0 ? -1 : to[tid];
        uint32_t x[4];
        if (r >= 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (w < words) x[w] = reinterpret_cast<const uint32_t*>(p + at(r, 4 * words))[w];
        }
        __syncthreads();
        if (d >= 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (w < words) reinterpret_cast<uint32_t*>(p + at(d, 4 * words))[w] = x[w];
        }
      }
    }
    if (n < kTokens) break;
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
  if (n == 0) return MK_OK;
  if (!src || !dst) return MK_ERR_INVALID;
  const mk_kv_pool& p = layers->pool;
  const bool q8 = p.kv_dtype == MK_KV_Q8;
  CopyArgs a{*layers, src, dst, n, 0, 0, static_cast<int64_t>(p.hkv) * kPage * p.dh * (q8 ? 1 : 2), static_cast<int64_t>(p.hkv) * p.dh};
  // 16 KB a block, or 4 KB where that leaves SMs without two blocks
  const bool big = a.page_bytes * 2 * n * layers->n_layers >= (304ll << 14);
  const int64_t span = kCopyBlock * 16 * (big ? 4 : 1);
  const int64_t chunks = (a.page_bytes + span - 1) / span, scale_chunks = q8 ? (a.scale_bytes + span - 1) / span : 0;
  if (2 * (chunks + scale_chunks) > 0x7fffffffll) return MK_ERR_UNSUPPORTED;
  a.chunks = static_cast<int>(chunks);
  a.scale_chunks = static_cast<int>(scale_chunks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (chunks + scale_chunks)), n < 65535 ? n : 65535, layers->n_layers);
  cfg.blockDim = dim3(kCopyBlock);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return launched(cudaLaunchKernelEx(&cfg, big ? kv_copy_kernel<4> : kv_copy_kernel<1>, a));
}

extern "C" mk_status mk_kv_keep(const mk_kv_layers* layers, const mk_kv_rows* rows, const int32_t* keep, int32_t* kv_len, void* stream) {
  using namespace mk::ops;
  mk_status st = check_layers(layers);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (rows->n_seqs == 0) return MK_OK;
  if (!keep && rows->n_rows > 0) return MK_ERR_INVALID;
  const mk_kv_pool& p = layers->pool;
  const bool q8 = p.kv_dtype == MK_KV_Q8;
  KeepArgs a{*layers, *rows, keep, kv_len, p.dh * (q8 ? 1 : 2), 0, 0, 1};
  const int64_t data = 2ll * p.hkv * (a.row_bytes / kWide), columns = data + (q8 ? 2ll * p.hkv : 0);
  if (columns > (1 << 24)) return MK_ERR_UNSUPPORTED;
  a.data = static_cast<int>(data);
  a.columns = static_cast<int>(columns);
  // as many columns a block as leave eight blocks an SM, up to eight
  const int64_t per = columns * rows->n_seqs * layers->n_layers / (152 * 8);
  a.per = per < 1 ? 1 : per > 8 ? 8 : static_cast<int>(per);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.columns + a.per - 1) / a.per), rows->n_seqs, layers->n_layers);
  cfg.blockDim = dim3(kTokens);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return launched(cudaLaunchKernelEx(&cfg, kv_keep_kernel, a));
}
