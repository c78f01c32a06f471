// Attention of a chunk of new rows over the paged cache: one warp per (row,
// query head), the online softmax over the tokens one by one.
#include <cuda_runtime.h>

#include <cmath>

#include "ops_internal.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kWarpsPerBlock = 4;

struct Args {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_attend_args a;
};

__device__ __forceinline__ float pool_value(const void* codes, const void* scale, int q8, int64_t e) {
  if (!q8) return __half2float(static_cast<const __half*>(codes)[e]);
  return __half2float(static_cast<const __half*>(scale)[e / 32]) * static_cast<float>(static_cast<const int8_t*>(codes)[e]);
}

template <int DT>
__global__ void attend_rows_kernel(const Args g) {
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + threadIdx.x / 32;
  if (w >= static_cast<int64_t>(g.rows.n_rows) * g.a.hq) return;
  const int r = static_cast<int>(w / g.a.hq), h = static_cast<int>(w % g.a.hq);
  int s = 0;
  SeqView v{0, 0, 0};
  for (; s < g.rows.n_seqs; ++s) {
    v = seq_view(g.rows, s);
    if (r >= v.r0 && r < v.r0 + v.q_len) break;
  }
  if (s == g.rows.n_seqs) return;
  const int pos = v.kv_len - v.q_len + (r - v.r0), dh = g.pool.dh, kh = h / (g.a.hq / g.pool.hkv);
  const int nd = dh / 32, q8 = g.pool.kv_dtype == MK_KV_Q8;
  float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
  const T* qp = static_cast<const T*>(g.a.q.data) + r * g.a.q.row_stride + h * g.a.q.head_stride;
  for (int i = 0; i < nd; ++i) q[i] = Elem<DT>::get(qp[32 * i + lane]) * g.a.scale;
  for (int t = 0; t <= pos; ++t) {
    if (g.a.window > 0 && pos - t >= g.a.window && t >= g.a.sinks) continue;
    const int page = g.rows.tables[static_cast<int64_t>(s) * g.rows.table_stride + t / kPage];
    if (page < 0 || page >= g.pool.n_pages) continue;
    const int64_t e = ((static_cast<int64_t>(page) * g.pool.hkv + kh) * kPage + t % kPage) * dh + lane;
    float x = 0.f;
    for (int i = 0; i < nd; ++i) x += q[i] * pool_value(g.pool.k, g.pool.k_scale, q8, e + 32 * i);
    for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    if (x == -INFINITY) continue;
    const float nm = fmaxf(m, x), f = expf(m - nm), p = expf(x - nm);
    m = nm;
    l = l * f + p;
    for (int i = 0; i < nd; ++i) o[i] = o[i] * f + p * pool_value(g.pool.v, g.pool.v_scale, q8, e + 32 * i);
  }
  for (int i = 0; i < nd; ++i) {
    float y = l > 0.f || l != l ? o[i] / l : 0.f;
    if (g.a.gate.data) {
      const T* gp = static_cast<const T*>(g.a.gate.data) + r * g.a.gate.row_stride + h * g.a.gate.head_stride;
      y /= 1.f + expf(-Elem<DT>::get(gp[32 * i + lane]));
    }
    static_cast<T*>(g.a.out.data)[r * g.a.out.row_stride + h * g.a.out.head_stride + 32 * i + lane] = Elem<DT>::put(y);
  }
}

mk_status check_attend(const mk_kv_pool* pool, const mk_kv_rows* rows, int32_t hq) {
  mk_status st = check_pool(pool);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (hq <= 0 || hq % pool->hkv) return MK_ERR_INVALID;
  return hq / pool->hkv > 256 ? MK_ERR_UNSUPPORTED : MK_OK;
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" size_t mk_attend_work_bytes(const mk_kv_pool* pool, const mk_kv_rows* rows, int32_t hq) {
  return mk::ops::check_attend(pool, rows, hq) == MK_OK ? 256 : 0;
}

extern "C" mk_status mk_attend(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_attend_args* a, void* stream) {
  using namespace mk::ops;
  if (!a) return MK_ERR_INVALID;
  const mk_status st = check_attend(pool, rows, a->hq);
  if (st != MK_OK) return st;
  if (a->dtype != MK_F16 && a->dtype != MK_BF16) return MK_ERR_INVALID;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale) || a->window < 0 || a->sinks < 0 || (a->sinks && !a->window))
    return MK_ERR_INVALID;
  if (!a->work || (reinterpret_cast<uintptr_t>(a->work) & 255u) || a->work_bytes < mk_attend_work_bytes(pool, rows, a->hq))
    return MK_ERR_INVALID;
  if (rows->n_seqs == 0 || rows->n_rows == 0) return MK_OK;
  if (!a->q.data || !a->out.data) return MK_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(a->q.data) | reinterpret_cast<uintptr_t>(a->out.data) |
        reinterpret_cast<uintptr_t>(a->gate.data)) & 1u))
    return MK_ERR_INVALID;
  const int64_t warps = static_cast<int64_t>(rows->n_rows) * a->hq;
  const int64_t grid = (warps + kWarpsPerBlock - 1) / kWarpsPerBlock;
  if (grid > 0x7fffffffll) return MK_ERR_UNSUPPORTED;
  const Args g{*pool, *rows, *a};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == MK_F16)
    attend_rows_kernel<MK_F16><<<static_cast<unsigned>(grid), kWarpsPerBlock * 32, 0, s>>>(g);
  else
    attend_rows_kernel<MK_BF16><<<static_cast<unsigned>(grid), kWarpsPerBlock * 32, 0, s>>>(g);
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
