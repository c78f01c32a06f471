// Write dense rows of K and V into the paged pool and read them back.
//
// One thread moves eight dims of one (row, kv head) of both K and V, so the
// row lookup is shared and two loads are in flight. Four neighbouring lanes
// hold one 32-dim q8 block (dh is a multiple of 64: a block never crosses a
// warp). Both kernels are bound by HBM traffic when there are many rows.
#include <cuda_runtime.h>

#include "ops_internal.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kBlock = 256;

struct RowsArgs {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_dense k, v;
  int row0, n;  // rows [row0, row0 + n) of this launch
};

struct Place {
  int64_t dense[2];  // element offset in the dense K and V
  int64_t elem;      // element offset in the pool, -1 none
  int r;
  bool live;  // the row belongs to a sequence
};

__device__ __forceinline__ bool place(const RowsArgs& a, int per_row, Place& p) {
  const uint32_t idx = blockIdx.x * static_cast<uint32_t>(kBlock) + threadIdx.x;
  const uint32_t n = static_cast<uint32_t>(a.n) * per_row;
  const int chunks = a.pool.dh / 8;
  const uint32_t i = min(idx, n - 1);  // lanes behind the end shadow the last chunk, without storing
  const int row = i / per_row, rest = i - row * per_row;
  const int head = rest / chunks, c = rest - head * chunks;
  p.r = a.row0 + row;
  p.dense[0] = p.r * a.k.row_stride + head * a.k.head_stride + c * 8;
  p.dense[1] = p.r * a.v.row_stride + head * a.v.head_stride + c * 8;
  const int t = token_row(a.rows, a.pool.n_pages, p.r);
  p.live = t != -2 && idx < n;
  // [page][head][slot][dh]
  p.elem = t < 0 ? -1
                 : ((static_cast<int64_t>(t / kPage) * a.pool.hkv + head) * kPage + t % kPage) * a.pool.dh + c * 8;
  return p.live;
}

template <int DT, bool Q8, bool VEC>
__global__ void __launch_bounds__(kBlock) kv_write_kernel(const RowsArgs a) {
  using T = typename Elem<DT>::T;
  Place p;
  const bool live = place(a, a.pool.hkv * (a.pool.dh / 8), p) && p.elem >= 0;
  float x[2][8] = {};
  if (live) {
    load8<DT, VEC>(static_cast<const T*>(a.k.data) + p.dense[0], x[0]);
    load8<DT, VEC>(static_cast<const T*>(a.v.data) + p.dense[1], x[1]);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    void* pool = w ? a.pool.v : a.pool.k;
    if (!Q8) {
      if (live) store8<MK_F16, true>(static_cast<__half*>(pool) + p.elem, x[w]);
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[w][i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const __half d16 = q8_scale(m);
    const float d = __half2float(d16), inv = __frcp_rn(d);
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo |= (static_cast<uint32_t>(q8_code(x[w][i], d, inv)) & 0xffu) << (8 * i);
      hi |= (static_cast<uint32_t>(q8_code(x[w][4 + i], d, inv)) & 0xffu) << (8 * i);
    }
    if (live) {
      *reinterpret_cast<uint2*>(static_cast<int8_t*>(pool) + p.elem) = make_uint2(lo, hi);
      if ((threadIdx.x & 3) == 0)
        static_cast<__half*>(w ? a.pool.v_scale : a.pool.k_scale)[p.elem / 32] = d16;
    }
  }
}

template <int DT, bool Q8, bool VEC>
__global__ void __launch_bounds__(kBlock) kv_read_kernel(const RowsArgs a) {
  using T = typename Elem<DT>::T;
  Place p;
  if (!place(a, a.pool.hkv * (a.pool.dh / 8), p)) return;
  float x[2][8] = {};
  if (p.elem >= 0) {
    if (!Q8) {
      load8<MK_F16, true>(static_cast<const __half*>(a.pool.k) + p.elem, x[0]);
      load8<MK_F16, true>(static_cast<const __half*>(a.pool.v) + p.elem, x[1]);
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(w ? a.pool.v : a.pool.k) + p.elem));
        const float d = __half2float(static_cast<const __half*>(w ? a.pool.v_scale : a.pool.k_scale)[p.elem / 32]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[w][i] = d * static_cast<float>(static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3))));
      }
    }
  }
  store8<DT, VEC>(static_cast<T*>(a.k.data) + p.dense[0], x[0]);
  store8<DT, VEC>(static_cast<T*>(a.v.data) + p.dense[1], x[1]);
}

using Kernel = void (*)(const RowsArgs);

template <bool WRITE, int DT>
Kernel pick_dt(bool q8, bool vec) {
  if (WRITE)
    return q8 ? (vec ? kv_write_kernel<DT, true, true> : kv_write_kernel<DT, true, false>)
              : (vec ? kv_write_kernel<DT, false, true> : kv_write_kernel<DT, false, false>);
  return q8 ? (vec ? kv_read_kernel<DT, true, true> : kv_read_kernel<DT, true, false>)
            : (vec ? kv_read_kernel<DT, false, true> : kv_read_kernel<DT, false, false>);
}

template <bool WRITE>
mk_status run(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_dense* k, const mk_dense* v, int32_t dtype,
              void* stream) {
  mk_status st = check_pool(pool);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (!k || !v || dtype < MK_F32 || dtype > MK_BF16) return MK_ERR_INVALID;
  if (rows->n_seqs == 0 || rows->n_rows == 0) return MK_OK;
  if (!k->data || !v->data) return MK_ERR_INVALID;
  const uintptr_t low = elem_bytes(dtype) - 1;
  if ((reinterpret_cast<uintptr_t>(k->data) & low) || (reinterpret_cast<uintptr_t>(v->data) & low)) return MK_ERR_INVALID;
  const bool vec = dense_vec(*k, dtype) && dense_vec(*v, dtype), q8 = pool->kv_dtype == MK_KV_Q8;
  const Kernel fn = dtype == MK_F32   ? pick_dt<WRITE, MK_F32>(q8, vec)
                    : dtype == MK_F16 ? pick_dt<WRITE, MK_F16>(q8, vec)
                                      : pick_dt<WRITE, MK_BF16>(q8, vec);
  const int64_t per_row = static_cast<int64_t>(pool->hkv) * (pool->dh / 8);
  if (per_row > (1 << 24)) return MK_ERR_UNSUPPORTED;
  const int slab = static_cast<int>((1ll << 30) / per_row);  // chunks of one launch stay below 2^31
  for (int64_t r = 0; r < rows->n_rows; r += slab) {
    RowsArgs a{*pool, *rows, *k, *v, static_cast<int>(r), static_cast<int>(rows->n_rows - r < slab ? rows->n_rows - r : slab)};
    const unsigned grid = static_cast<unsigned>((a.n * per_row + kBlock - 1) / kBlock);
    fn<<<grid, kBlock, 0, static_cast<cudaStream_t>(stream)>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_kv_write(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_dense* k, const mk_dense* v,
                                 int32_t dtype, void* stream) {
  return mk::ops::run<true>(pool, rows, k, v, dtype, stream);
}

extern "C" mk_status mk_kv_read(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_dense* k, const mk_dense* v,
                                int32_t dtype, void* stream) {
  return mk::ops::run<false>(pool, rows, k, v, dtype, stream);
}
