// Greedy verification of a tree of drafts.
//
// Each node's greedy token g is the argmax of its logits (the lowest index where
// several are largest). The path starts at a sequence's first row and goes on to the
// lowest child whose draft token is g of the node it has reached. Children lie behind
// their parents, so one scan of the nodes finds it.
//
// Two launches: tree_top takes the maximum of a row's part per block, tree_walk (launched
// early) joins the parts and walks, a block per sequence. Where a sequence's logits are few,
// tree_small does both in one launch. Bound by the logits' bytes when the vocabulary is large,
// by the launches when it is small. 64 rows of 248,320 fp32 logits (64 MB): 15 us, of which
// tree_top takes 12 (5.3 TB/s) and tree_walk 3 (the parts' latency); of 16-bit logits (32 MB) 16
// to 17 us in replayed graphs, where fp32 takes 18.5: as many comparisons (issue slots 48 %
// active, DRAM at 28 %). 8 rows of 2,048: 7 us through Python.
#include <climits>

#include <cuda_runtime.h>

#include "ops_internal.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxSplit = 128;  // parts of a row
constexpr int kSpan = 2048;     // logits of a part, at least
constexpr int kMaxVocab = 1 << 30;  // indices of a row's parts stay within 32 bits
constexpr int64_t kSmall = 1 << 15;
constexpr int kSmallVocab = 1 << 12;

// A logit and its index as one number that grows with the logit and falls with the
// index; a NaN is above every number.
constexpr uint64_t kNan = ~0ull;
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // (-0 is 0)
  return static_cast<uint64_t>(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int token_of(uint64_t key) {
  return key == kNan || key == 0 ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, k, m);
    k = o > k ? o : k;
  }
  return k;
}

struct TreeArgs {
  mk_kv_rows rows;
  const int32_t* parents;
  const int32_t* tokens;
  const void* logits;
  int64_t row_stride;
  int vocab, split, span;  // parts of a row, logits of a part
  int32_t* path;
  int32_t* count;
  int32_t* emitted;
  uint64_t* part;  // [rows][split]
  int32_t* greedy;  // [rows]
};

// The largest of logits [i0, end) that a thread of `threads` sees, 16 bytes at a time from its own first ones on, as a key
// (0: it sees none). Ascending, so that the first of equal ones stays.
template <int DT, bool VEC>
__device__ __forceinline__ uint64_t scan(const typename Elem<DT>::T* x, int begin, int end, int thread, int threads) {
  using T = typename Elem<DT>::T;
  constexpr int kV = 16 / sizeof(T), kDeep = 8;
  const int step = threads * kV, i0 = begin + thread * kV;
  float best = -INFINITY;
  int at = INT_MAX;
  bool nan = false;
  auto see = [&](float y, int i) {
    if (!(y <= best)) {  // larger, or a NaN
      nan |= y != y;
      best = y;
      at = i;
    }
  };
  auto get = [&](int j, float* y) {
    if (VEC) {
      const uint4 w = *reinterpret_cast<const uint4*>(x + j);
#pragma unroll
      for (int k = 0; k < kV; ++k) y[k] = Elem<DT>::get(reinterpret_cast<const T*>(&w)[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kV; ++k) y[k] = Elem<DT>::get(x[j + k]);
    }
  };
  int i = i0;
  for (; i + (kDeep - 1) * step + kV <= end; i += kDeep * step) {
    float y[kDeep][kV];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) get(i + u * step, y[u]);
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
#pragma unroll
      for (int k = 0; k < kV; ++k) see(y[u][k], i + u * step + k);
  }
  for (; i + kV <= end; i += step) {
    float y[kV];
    get(i, y);
#pragma unroll
    for (int k = 0; k < kV; ++k) see(y[k], i + k);
  }
  for (; i < end; ++i) see(Elem<DT>::get(x[i]), i);
  return nan ? kNan : at != INT_MAX ? key_of(best, at) : i0 < end ? key_of(-INFINITY, i0) : 0;
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kBlock) tree_top(const __grid_constant__ TreeArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ uint64_t top[kBlock / 32];
  let_next_start();  // tree_walk
  wait_for_previous();
  for (int row = blockIdx.y; row < a.rows.n_rows; row += gridDim.y) {
    const int begin = static_cast<int>(blockIdx.x) * a.span;
    uint64_t key = scan<DT, VEC>(static_cast<const T*>(a.logits) + row * a.row_stride, begin, min(a.vocab, begin + a.span),
                                 threadIdx.x, kBlock);
    key = warp_max(key);
    if ((threadIdx.x & 31) == 0) top[threadIdx.x / 32] = key;
    __syncthreads();
    if (threadIdx.x < 32) {
      key = warp_max(threadIdx.x < kBlock / 32 ? top[threadIdx.x] : 0);
      if (threadIdx.x == 0) a.part[static_cast<int64_t>(row) * a.split + blockIdx.x] = key;
    }
    __syncthreads();
  }
}

// A warp walks a sequence's tree, 32 nodes at a time; greedy: its nodes' greedy tokens.
template <class Greedy>
__device__ __forceinline__ void walk(const TreeArgs& a, const SeqView& v, int seq, int lane, Greedy greedy) {
  int count = 0, cur = 0, want = -1;
  auto reach = [&](int node) {
    cur = node;
    want = greedy(node);
    if (lane == 0) {
      a.path[v.r0 + count] = node;
      a.emitted[v.r0 + count] = want;
    }
    ++count;
  };
  int parent = -1, tok = -1;
  auto fetch = [&](int j) {
    if (j < v.q_len) {
      parent = a.parents ? parent_of(a.parents + v.r0, j) : j - 1;
      tok = a.tokens[v.r0 + j];
    }
  };
  fetch(1 + lane);
  if (v.q_len) reach(0);
  for (int j0 = 1; j0 < v.q_len; j0 += 32) {
    const int j = j0 + lane;
    if (j0 > 1) fetch(j);
    for (;;) {  // (each hit lies behind the one before: no more than 32)
      const uint32_t hit = __ballot_sync(0xffffffffu, j < v.q_len && parent == cur && want >= 0 && tok == want);
      if (!hit) break;
      reach(j0 + __ffs(hit) - 1);
    }
  }
  for (int j = count + lane; j < v.q_len; j += 32) {
    a.path[v.r0 + j] = -1;
    a.emitted[v.r0 + j] = -1;
  }
  if (lane == 0) a.count[seq] = count;
}

constexpr int kWalkBlock = 512, kNear = 1024;  // nodes whose greedy tokens are kept in shared memory

__global__ void __launch_bounds__(kWalkBlock) tree_walk(const __grid_constant__ TreeArgs a) {
  __shared__ int near[kNear];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();  // the parts are there from here on
  const SeqView v = seq_view(a.rows, blockIdx.x);
  for (int j = warp; j < v.q_len; j += kWalkBlock / 32) {
    uint64_t key = 0;
    for (int p = lane; p < a.split; p += 32) {
      const uint64_t o = a.part[static_cast<int64_t>(v.r0 + j) * a.split + p];
      key = o > key ? o : key;
    }
    key = warp_max(key);
    if (lane == 0) (j < kNear ? near[j] : a.greedy[v.r0 + j]) = token_of(key);
  }
  __syncthreads();
  if (warp == 0) walk(a, v, blockIdx.x, lane, [&](int j) { return j < kNear ? near[j] : a.greedy[v.r0 + j]; });
}

// A block takes a whole sequence, a warp a row at a time.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kWalkBlock) tree_small(const __grid_constant__ TreeArgs a) {
  using T = typename Elem<DT>::T;
  __shared__ int near[kNear];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();
  const SeqView v = seq_view(a.rows, blockIdx.x);
  for (int j = warp; j < v.q_len; j += kWalkBlock / 32) {
    const uint64_t key = warp_max(scan<DT, VEC>(static_cast<const T*>(a.logits) + (v.r0 + j) * a.row_stride, 0, a.vocab, lane, 32));
    if (lane == 0) near[j] = token_of(key);  // (no more rows than kNear)
  }
  __syncthreads();
  if (warp == 0) walk(a, v, blockIdx.x, lane, [&](int j) { return near[j]; });
}

// Parts of a row: about four blocks an SM over all rows, each of at least kSpan logits. (64 rows of 248,320 fp32 logits, eight
// loads a thread at a time: four blocks 16.6 us, five 17.7, eight 17.3; four loads: eight blocks 17.6.)
int split_of(int n_rows, int vocab) {
  const int64_t most = (static_cast<int64_t>(vocab) + kSpan - 1) / kSpan, want = (608 + n_rows - 1) / (n_rows > 0 ? n_rows : 1);
  const int64_t n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n > kMaxSplit ? kMaxSplit : n);
}
int64_t part_bytes(int n_rows, int vocab) { return (static_cast<int64_t>(n_rows) * split_of(n_rows, vocab) * 8 + 255) / 256 * 256; }

// One launch while the rows of a sequence (as many as max_q says) hold no more logits than kSmall, and a row, which one warp
// reads, no more than kSmallVocab (8 rows of 2,048: 3.1 against 3.4 us, 16 rows 3.8 against 3.9, 32 rows 6.0 against 4.6, 8 rows
// of 8,192 6.7 against 3.8; besides, it spares the host a launch). Its nodes' greedy tokens stay in shared memory: no workspace.
bool small(const mk_kv_rows& rows, int vocab) {
  return rows.n_rows <= kNear && vocab <= kSmallVocab && static_cast<int64_t>(rows.max_q) * vocab <= kSmall;
}

template <int DT>
cudaError_t launch(const TreeArgs& a, bool vec, cudaStream_t stream) {
  if (small(a.rows, a.vocab))
    return launch_early(vec ? tree_small<DT, true> : tree_small<DT, false>, dim3(a.rows.n_seqs), dim3(kWalkBlock), 0, stream, a);
  const dim3 grid(a.split, a.rows.n_rows < 65535 ? a.rows.n_rows : 65535);
  const cudaError_t e = launch_early(vec ? tree_top<DT, true> : tree_top<DT, false>, grid, dim3(kBlock), 0, stream, a);
  return e != cudaSuccess ? e : launch_early(tree_walk, dim3(a.rows.n_seqs), dim3(kWalkBlock), 0, stream, a);
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" size_t mk_tree_work_bytes(const mk_kv_rows* rows, int32_t vocab) {
  using namespace mk::ops;
  if (check_rows(rows) != MK_OK || rows->n_rows > kMaxList || vocab <= 0 || vocab > kMaxVocab || small(*rows, vocab)) return 0;
  return static_cast<size_t>(part_bytes(rows->n_rows, vocab)) + static_cast<size_t>(rows->n_rows) * 4 + 256;
}

extern "C" mk_status mk_tree_accept(const mk_kv_rows* rows, const mk_tree_args* t, void* stream) {
  using namespace mk::ops;
  const mk_status st = check_rows(rows);
  if (st != MK_OK) return st;
  if (!t || t->vocab <= 0 || t->dtype < MK_F32 || t->dtype > MK_BF16) return MK_ERR_INVALID;
  if (t->vocab > kMaxVocab || rows->n_rows > kMaxList) return MK_ERR_UNSUPPORTED;
  if (rows->n_seqs == 0) return MK_OK;
  if (!t->count) return MK_ERR_INVALID;
  if (rows->n_rows > 0) {
    if (!t->tokens || !t->logits || !t->path || !t->emitted || (reinterpret_cast<uintptr_t>(t->logits) & (elem_bytes(t->dtype) - 1)))
      return MK_ERR_INVALID;
    const size_t need = mk_tree_work_bytes(rows, t->vocab);
    if (need && (!t->work || (reinterpret_cast<uintptr_t>(t->work) & 255u) || t->work_bytes < need)) return MK_ERR_INVALID;
  }
  TreeArgs a{*rows, t->parents, t->tokens, t->logits, t->row_stride, t->vocab, 1, 0, t->path, t->count, t->emitted, nullptr, nullptr};
  a.split = split_of(rows->n_rows, t->vocab);
  a.span = static_cast<int>(((static_cast<int64_t>(t->vocab) + a.split - 1) / a.split + 7) / 8 * 8);
  a.part = static_cast<uint64_t*>(t->work);
  a.greedy = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(t->work) + part_bytes(rows->n_rows, t->vocab));
  const bool vec = dense_vec(mk_dense{const_cast<void*>(t->logits), t->row_stride, 0}, t->dtype);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (rows->n_rows == 0) {  // no path anywhere
    e = cudaMemsetAsync(t->count, 0, sizeof(int32_t) * rows->n_seqs, s);
  } else {
    e = t->dtype == MK_F32 ? launch<MK_F32>(a, vec, s) : t->dtype == MK_F16 ? launch<MK_F16>(a, vec, s) : launch<MK_BF16>(a, vec, s);
  }
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}
