// Write dense rows of K and V into the paged pool and read them back.
//
// One thread moves twice eight dims, from the two halves of one (row, kv head),
// of both K and V: the row lookup is shared, four 16-byte loads (of 16-bit
// values) are in flight, and neighbouring lanes move neighbouring bytes. (16
// neighbouring dims a thread left gaps between the lanes' accesses.) Four
// neighbouring lanes hold two 32-dim q8 blocks (dh is a multiple of 64: a block
// never crosses a warp). Both kernels are bound by HBM traffic when there are
// many rows, by the launch when there are few. The dense rows are fetched
// before the lookup, whose three dependent loads would otherwise come first.
// 92,000 rows of 4 heads of 256 (bf16): write 114 us to fp16 (6.6 TB/s), 141 us
// to q8 (615 instructions a warp); read 123 us from fp16, 102 us from q8.
#include <cuda_runtime.h>

#include "ops_internal.cuh"
#include "q8_codec.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kBlock = 256;

struct RowsArgs {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_dense k, v;
  int row0, n;       // rows [row0, row0 + n) of this launch
  uint32_t per_row;  // threads a row: kv heads x dh / 16
  uint32_t inv;      // floor(2^32 / per_row)
};

// Thread's row (live), head and first eight dims; the others are dh / 2 on.
// Threads behind the end shadow the last row without storing.
struct Where {
  int64_t r;
  int head, dim;
  bool live;
};
__device__ __forceinline__ Where where(const RowsArgs& a) {
  const uint32_t idx = blockIdx.x * static_cast<uint32_t>(kBlock) + threadIdx.x;
  uint32_t g = __umulhi(idx, a.inv);  // idx / per_row or one less
  uint32_t rest = idx - g * a.per_row;
  if (rest >= a.per_row) {
    rest -= a.per_row;
    ++g;
  }
  const uint32_t chunks = static_cast<uint32_t>(a.pool.dh) / 16;
  const int head = rest / chunks;
  Where w;
  w.live = g < static_cast<uint32_t>(a.n);
  w.r = a.row0 + (w.live ? static_cast<int>(g) : a.n - 1);
  w.head = head;
  w.dim = static_cast<int>(rest - head * chunks) * 8;
  return w;
}
// [page][head][slot][dh]
__device__ __forceinline__ int64_t pool_elem(const RowsArgs& a, int token_row, const Where& w) {
  return ((static_cast<int64_t>(token_row / kPage) * a.pool.hkv + w.head) * kPage + token_row % kPage) * a.pool.dh + w.dim;
}

template <int DT, bool Q8, bool VEC>
__global__ void __launch_bounds__(kBlock, 5) kv_write_kernel(const RowsArgs a) {
  using T = typename Elem<DT>::T;
  wait_for_previous();
  const Where w = where(a);
  const int half = a.pool.dh / 2;
  const T* k = static_cast<const T*>(a.k.data) + w.r * a.k.row_stride + w.head * a.k.head_stride + w.dim;
  const T* v = static_cast<const T*>(a.v.data) + w.r * a.v.row_stride + w.head * a.v.head_stride + w.dim;
  float x[4][8];
  load8<DT, VEC>(k, x[0]);
  load8<DT, VEC>(k + half, x[1]);
  load8<DT, VEC>(v, x[2]);
  load8<DT, VEC>(v + half, x[3]);
  const int t = w.live ? token_row(a.rows, a.pool.n_pages, static_cast<int>(w.r)) : -1;
  const int64_t elem = t < 0 ? 0 : pool_elem(a, t, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    void* pool = i < 2 ? a.pool.k : a.pool.v;
    const int64_t e = elem + (i & 1) * half;
    if (!Q8) {
      if (t >= 0) store8<MK_F16, true>(static_cast<__half*>(pool) + e, x[i]);
      continue;
    }
    float m = fabsf(x[i][0]);  // (a block of NaN alone has a NaN scale)
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(x[i][j]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // four lanes hold a block of 32
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float d = q8_scale(m);
    uint32_t c[2];
    q8_codes<8>(x[i], d, m, c);
    if (t >= 0) {
      *reinterpret_cast<uint2*>(static_cast<int8_t*>(pool) + e) = make_uint2(c[0], c[1]);
      if ((threadIdx.x & 3) == 0)
        static_cast<__half*>(i < 2 ? a.pool.k_scale : a.pool.v_scale)[e / 32] = __float2half_rn(d);
    }
  }
}

template <int DT, bool Q8, bool VEC>
__global__ void __launch_bounds__(kBlock) kv_read_kernel(const RowsArgs a) {
  using T = typename Elem<DT>::T;
  wait_for_previous();
  const Where w = where(a);
  const int t = w.live ? token_row(a.rows, a.pool.n_pages, static_cast<int>(w.r)) : -2;
  if (t == -2) return;
  const int half = a.pool.dh / 2;
  float x[4][8] = {};
  if (t >= 0) {
    const int64_t elem = pool_elem(a, t, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const void* pool = i < 2 ? a.pool.k : a.pool.v;
      const int64_t e = elem + (i & 1) * half;
      if (!Q8) {
        load8<MK_F16, true>(static_cast<const __half*>(pool) + e, x[i]);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(pool) + e);
        const float d = __half2float(static_cast<const __half*>(i < 2 ? a.pool.k_scale : a.pool.v_scale)[e / 32]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // 2^23 + (code + 128) by a byte move: integer conversions run at a quarter of the rate
          const uint32_t w = (j < 4 ? c.x : c.y) ^ 0x80808080u;
          x[i][j] = d * (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 | (j & 3))) - 8388736.0f);
        }
      }
    }
  }
  T* k = static_cast<T*>(a.k.data) + w.r * a.k.row_stride + w.head * a.k.head_stride + w.dim;
  T* v = static_cast<T*>(a.v.data) + w.r * a.v.row_stride + w.head * a.v.head_stride + w.dim;
  store8<DT, VEC>(k, x[0]);
  store8<DT, VEC>(k + half, x[1]);
  store8<DT, VEC>(v, x[2]);
  store8<DT, VEC>(v + half, x[3]);
}

using Kernel = void (*)(const RowsArgs);

template <bool WRITE, int DT>
Kernel pick(bool q8, bool vec) {
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
  const int64_t per_row = static_cast<int64_t>(pool->hkv) * (pool->dh / 16);
  if (per_row > (1 << 24)) return MK_ERR_UNSUPPORTED;
  const Kernel fn = dtype == MK_F32   ? pick<WRITE, MK_F32>(q8, vec)
                    : dtype == MK_F16 ? pick<WRITE, MK_F16>(q8, vec)
                                      : pick<WRITE, MK_BF16>(q8, vec);
  const int64_t slab = (1ll << 30) / per_row;  // threads of one launch stay below 2^31
  for (int64_t r = 0; r < rows->n_rows; r += slab) {
    RowsArgs a{*pool, *rows, *k, *v, static_cast<int>(r),
               static_cast<int>(rows->n_rows - r < slab ? rows->n_rows - r : slab), static_cast<uint32_t>(per_row),
               static_cast<uint32_t>((1ll << 32) / per_row)};
    const dim3 grid(static_cast<unsigned>((a.n * per_row + kBlock - 1) / kBlock));
    if (launch_early(fn, grid, dim3(kBlock), 0, static_cast<cudaStream_t>(stream), a) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
  }
  return MK_OK;
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
