// Shared by the KV-cache operators: argument checks, the row map, and
// typed loads and stores of eight elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mk_ops.h"

namespace mk {
namespace ops {

constexpr int kPage = 16;

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

inline int elem_bytes(int dtype) { return dtype == MK_F32 ? 4 : 2; }

// Whether eight elements can be moved with 16-byte accesses.
inline bool dense_vec(const mk_dense& d, int dtype) {
  const int per = 16 / elem_bytes(dtype);
  return aligned16(d.data) && d.row_stride % per == 0 && d.head_stride % per == 0;
}

// ----------------------------------------------------------------- row map
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

struct SeqView {
  int r0, q_len, kv_len;  // first row, rows, tokens; all within bounds
};
__device__ __forceinline__ SeqView seq_view(const mk_kv_rows& m, int s) {
  SeqView v;
  v.r0 = clampi(__ldg(m.row_start + s), 0, m.n_rows);
  v.q_len = clampi(__ldg(m.row_start + s + 1), v.r0, m.n_rows) - v.r0;
  v.kv_len = clampi(__ldg(m.kv_len + s), 0, m.table_stride * kPage);
  return v;
}

// Token row (page * 16 + slot) of dense row r, -1 when it has none, -2 when r
// belongs to no sequence. The sequence is the first whose end lies behind r.
__device__ __forceinline__ int token_row(const mk_kv_rows& m, int n_pages, int r) {
  int lo = 0, hi = m.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(m.row_start + mid + 1) > r) hi = mid; else lo = mid + 1;
  }
  if (lo >= m.n_seqs) return -2;
  const SeqView v = seq_view(m, lo);
  if (r < v.r0 || r >= v.r0 + v.q_len) return -2;
  const int pos = v.kv_len - v.q_len + (r - v.r0);
  if (pos < 0) return -1;
  const int page = __ldg(m.tables + static_cast<int64_t>(lo) * m.table_stride + pos / kPage);
  return page >= 0 && page < n_pages ? page * kPage + pos % kPage : -1;
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
      reinterpret_cast<uint4*>(t)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
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
