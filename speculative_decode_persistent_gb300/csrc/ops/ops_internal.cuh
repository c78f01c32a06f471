// Shared by the KV-cache operators: argument checks, the row map, and
// typed loads and stores of eight elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mk_ops.h"

namespace mk {
namespace ops {

constexpr int kPage = 16;
// Entries of a list, or rows, that a kernel steps through in strides of up to 2^17: the next index stays within 32 bits.
constexpr int kMaxList = 1 << 30;

// ------------------------------------------------------------- host checks
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline mk_status check_pool(const mk_kv_pool* p) {
  if (!p || !p->k || !p->v || p->n_pages <= 0 || p->hkv <= 0 || p->dh <= 0) return MK_ERR_INVALID;
  if (p->kv_dtype != MK_KV_F16 && p->kv_dtype != MK_KV_Q8) return MK_ERR_INVALID;
  if (!aligned16(p->k) || !aligned16(p->v)) return MK_ERR_INVALID;
  if (p->kv_dtype == MK_KV_Q8 &&
      (!p->k_scale || !p->v_scale || !aligned16(p->k_scale) || !aligned16(p->v_scale)))
    return MK_ERR_INVALID;
  if (p->dh % 64 || p->dh > 256) return MK_ERR_UNSUPPORTED;
  // token rows of the pool are addressed with 32 bits (times dh: with 64)
  if (static_cast<int64_t>(p->n_pages) * p->hkv * kPage > 0x7fffffffll) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

inline mk_status check_rows(const mk_kv_rows* r) {
  if (!r || r->n_seqs < 0 || r->n_rows < 0 || r->table_stride < 0) return MK_ERR_INVALID;
  if (r->n_seqs > 0 && (!r->row_start || !r->kv_len || (!r->tables && r->table_stride > 0))) return MK_ERR_INVALID;
  if (r->n_seqs > MK_OPS_MAX_SEQS || r->table_stride > 0x7fffffff / kPage) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

inline mk_status check_layers(const mk_kv_layers* l) {
  if (!l) return MK_ERR_INVALID;
  const mk_status st = check_pool(&l->pool);
  if (st != MK_OK) return st;
  const int64_t layer = static_cast<int64_t>(l->pool.n_pages) * l->pool.hkv * kPage * l->pool.dh;
  // (a multiple of 256 elements keeps every layer's scales on 16 bytes)
  if (l->n_layers <= 0 || (l->n_layers > 1 && (l->layer_stride < layer || l->layer_stride % 256))) return MK_ERR_INVALID;
  return l->n_layers > 65535 ? MK_ERR_UNSUPPORTED : MK_OK;
}

inline int elem_bytes(int dtype) { return dtype == MK_F32 ? 4 : 2; }

// Whether eight elements can be moved with 16-byte accesses.
inline bool dense_vec(const mk_dense& d, int dtype) {
  const int per = 16 / elem_bytes(dtype);
  return aligned16(d.data) && d.row_stride % per == 0 && d.head_stride % per == 0;
}

// ------------------------------------------------------------ early launches
// Kernels are launched while the one before them in the stream ends: their launch overlaps its end (tree of 8 nodes over
// 4K tokens 20.5 -> 17.5 us a call, 64 rotated rows 11.9 -> 10.5). The first thing every thread does with memory that
// others use is to wait for that end, so a kernel is over only after all those before it. What it reads then it reads with
// ordinary loads, which the wait orders: read-only ones (ld.global.nc) promise the right value only of memory that nothing
// writes while the kernel runs, and it runs while the one before still writes. A kernel lets the next one in
// before its end only where that is its own second part: another kernel's blocks, placed among those still running,
// would lie unevenly on the SMs (kept tokens 132 -> 152 us).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};  // (the launch's own status: an error that an earlier call left is not this one's)
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ----------------------------------------------------------------- row map
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

struct SeqView {
  int r0, q_len, kv_len;  // first row, rows, tokens; all within bounds
};
__device__ __forceinline__ SeqView seq_view(const mk_kv_rows& m, int s) {
  SeqView v;
  v.r0 = clampi(m.row_start[s], 0, m.n_rows);
  v.q_len = clampi(m.row_start[s + 1], v.r0, m.n_rows) - v.r0;
  v.kv_len = clampi(m.kv_len[s], 0, m.table_stride * kPage);
  return v;
}

// Token row (page * 16 + slot) of position pos of sequence s, -1 when it has none.
__device__ __forceinline__ int token_at(const mk_kv_rows& m, int n_pages, int s, int pos) {
  if (pos < 0 || pos >= m.table_stride * kPage) return -1;
  const int page = m.tables[static_cast<int64_t>(s) * m.table_stride + pos / kPage];
  return page >= 0 && page < n_pages ? page * kPage + pos % kPage : -1;
}

// Sequence of dense row r, the first whose end lies behind r, and its view; -1 when r belongs to none.
__device__ __forceinline__ int seq_of_row(const mk_kv_rows& m, int r, SeqView& v) {
  int lo = 0, hi = m.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (m.row_start[mid + 1] > r) hi = mid; else lo = mid + 1;
  }
  if (lo >= m.n_seqs) return -1;
  v = seq_view(m, lo);
  return r < v.r0 || r >= v.r0 + v.q_len ? -1 : lo;
}

// Token row of dense row r, -1 when it has none, -2 when r belongs to no sequence.
__device__ __forceinline__ int token_row(const mk_kv_rows& m, int n_pages, int r) {
  SeqView v;
  const int s = seq_of_row(m, r, v);
  return s < 0 ? -2 : token_at(m, n_pages, s, v.kv_len - v.q_len + (r - v.r0));
}

// A node's parent in a tree of drafts (parents: of its sequence's rows), -1 for none: only a node before it can be one,
// so every walk towards the root ends.
__device__ __forceinline__ int parent_of(const int32_t* parents, int node) {
  const int p = parents[node];
  return p >= 0 && p < node ? p : -1;
}

// ------------------------------------------------------------- eight values
template <int DT>
struct Elem;
template <>
struct Elem<MK_F32> {
  using T = float;
  static __device__ float get(T x) { return x; }
  static __device__ T put(float x) { return x; }
};
template <>
struct Elem<MK_F16> {
  using T = __half;
  static __device__ float get(T x) { return __half2float(x); }
  static __device__ T put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<MK_BF16> {
  using T = __nv_bfloat16;
  static __device__ float get(T x) { return __bfloat162float(x); }
  static __device__ T put(float x) { return __float2bfloat16_rn(x); }
};

template <int DT, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* p, float* x) {
  using T = typename Elem<DT>::T;
  alignas(16) T t[8];
  if (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::get(t[i]);
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float* x) {
  using T = typename Elem<DT>::T;
  alignas(16) T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = Elem<DT>::put(x[i]);
  if (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(t)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = t[i];
  }
}

}  // namespace ops
}  // namespace mk
