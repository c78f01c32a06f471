// C entry of the chunk attention: argument checks, tensor maps of the pool,
// choice of the kernel.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "attend.cuh"

namespace mk {
namespace ops {
using Launch = cudaError_t(int ns, int cg, const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv, int device,
                           cudaStream_t stream);
Launch launch_attend_f16, launch_attend_q8, launch_attend_tree_f16, launch_attend_tree_q8;

namespace {

mk_status check_attend(const mk_kv_pool* pool, const mk_kv_rows* rows, int32_t hq) {
  mk_status st = check_pool(pool);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (hq <= 0 || hq % pool->hkv) return MK_ERR_INVALID;
  if (hq / pool->hkv > 256) return MK_ERR_UNSUPPORTED;
  // (row, head) pairs, and the blocks of all tiles, are counted with 32 bits
  if (static_cast<int64_t>(rows->n_rows) * hq > 0x7fff0000ll) return MK_ERR_UNSUPPORTED;
  const double tiles = static_cast<double>(rows->n_rows) * hq / 128 + static_cast<double>(rows->n_seqs) * pool->hkv;
  return tiles * (rows->table_stride / (kBN / kPage) + 2 + item_cost(256)) > 2e9 ? MK_ERR_UNSUPPORTED : MK_OK;
}

// Test hook (mk_debug_attend_wait).
constexpr int kWaitUs = 2000000;
std::atomic<int> g_wait_us{kWaitUs}, g_skip{-1};

constexpr size_t kJoinBytes = (kMaxWorkers * sizeof(JoinInfo) + 255) / 256 * 256;
// two parts per worker of 128 rows a block
constexpr size_t kMlBytes = 2ull * kMaxWorkers * 128 * sizeof(float2);

// The pool as token rows of dh elements. binary16: [slab of 64][token][64],
// boxes of `slabs` x `tokens` rows of 128 bytes, swizzled as the products read
// them. q8: boxes of 16 tokens x `box` codes.
bool encode_map(CUtensorMap* m, void* base, const mk_kv_pool& p, int box, int tokens, int slabs) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dh = static_cast<cuuint64_t>(p.dh), rows = static_cast<cuuint64_t>(p.n_pages) * p.hkv * kPage;
  const cuuint32_t one[3] = {1, 1, 1};
  if (p.kv_dtype == MK_KV_Q8) {
    const cuuint64_t dims[2] = {dh, rows}, strides[1] = {dh};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), kPage};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[3] = {64, rows, dh / 64}, strides[2] = {dh * 2, 128};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(tokens), static_cast<cuuint32_t>(slabs)};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" size_t mk_attend_work_bytes(const mk_kv_pool* pool, const mk_kv_rows* rows, int32_t hq) {
  using namespace mk::ops;
  if (check_attend(pool, rows, hq) != MK_OK) return 0;
  return kJoinBytes + kMlBytes + 2ull * kMaxWorkers * 128 * pool->dh * sizeof(float);
}

extern "C" mk_status mk_debug_attend_wait(int32_t wait_us, int32_t skip_worker) {
  if (wait_us < 0 || wait_us > mk::ops::kWaitUs || skip_worker < -1) return MK_ERR_INVALID;
  mk::ops::g_wait_us.store(wait_us ? wait_us : mk::ops::kWaitUs);
  mk::ops::g_skip.store(skip_worker);
  return MK_OK;
}

extern "C" mk_status mk_attend(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_attend_args* a, void* stream) {
  return mk_attend_tree(pool, rows, a, nullptr, stream);
}

extern "C" mk_status mk_attend_tree(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_attend_args* a, const int32_t* parents,
                                    void* stream) {
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

  AttendParams p{};
  p.pool = *pool;
  p.rows = *rows;
  p.q = a->q;
  p.gate = a->gate;
  p.out = a->out;
  p.hq = a->hq;
  p.G = a->hq / pool->hkv;
  p.g_inv = (1 << 20) / p.G + 1;
  p.dtype = a->dtype;
  p.parents = parents;
  // a window beyond every length is none, and keeps the positions' arithmetic in range
  p.window = a->window >= rows->table_stride * kPage ? 0 : a->window;
  p.sinks = p.window ? a->sinks : 0;
  p.c = std::fmin(std::fmax(a->scale * 1.44269504088896341f, 1.2e-38f), 3e38f);
  p.vq = dense_vec(a->q, a->dtype);
  p.vo = dense_vec(a->out, a->dtype);
  if (p.vo && reinterpret_cast<uintptr_t>(a->out.data) % 32 == 0 && a->out.row_stride % 16 == 0 && a->out.head_stride % 16 == 0)
    p.vo = 2;
  p.vg = dense_vec(a->gate, a->dtype);
  p.wait_us = g_wait_us.load();
  p.skip = g_skip.load();
  uint8_t* w = static_cast<uint8_t*>(a->work);
  p.join = reinterpret_cast<JoinInfo*>(w);
  p.ml = reinterpret_cast<float2*>(w + kJoinBytes);
  p.part = reinterpret_cast<float*>(w + kJoinBytes + kMlBytes);

  const int ns = pool->dh / 64, q8 = pool->kv_dtype == MK_KV_Q8;
  // Pairs of blocks where a sequence fills more than one 128-row tile: they
  // fetch half the bytes per product. Below that the second block of a pair
  // would have no rows, and single blocks keep twice as many copies going.
  const int cg = ns % 2 == 0 && static_cast<int64_t>(rows->max_q) * p.G > 128 ? 2 : 1;
  CUtensorMap tk, tv;
  const int box = q8_box(ns, cg), slabs_k = ns, slabs_v = ns / cg;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || !encode_map(&tk, pool->k, *pool, box, slabs_k == 1 ? kPage : 8, slabs_k) ||
      !encode_map(&tv, pool->v, *pool, box, kPage, slabs_v))
    return MK_ERR_CUDA;
  Launch* const launch = parents ? (q8 ? launch_attend_tree_q8 : launch_attend_tree_f16) : q8 ? launch_attend_q8 : launch_attend_f16;
  const cudaError_t e = launch(ns, cg, p, tk, tv, device, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}
