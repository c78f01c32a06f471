// Norm, position rotation and write of new rows in one pass.
//
// Mathematics. A q or k head vector x is scaled to y = x (mean x^2 + eps)^-1/2 g
// (when there are gains), then y_i and y_{i + r/2}, i < r/2, are turned by the
// angle p f_i, p the row's position and f_i its pair's frequency. q goes to a dense
// tensor, k and v to their slots of the pool, rounded once or quantised.
//
// Angles. A 32-bit product p f_i is off by p 2^-24 radians, and 64-bit floating
// point runs at a 64th of the rate. f_i / 2 pi is therefore kept as a 64-bit
// fraction of a turn, and p times it, modulo 2^64, is the angle in turns up to
// p 2^-65: a few integer products. Its upper 32 bits, as half turns in (-1, 1), go
// into sincospif.
//
// Layout. dh / 16 neighbouring lanes hold a head vector, eight dims and the
// eight that they are paired with per lane (dims that are not turned are paired
// the same way): the turn stays in the thread, the norm's sum takes up to four
// shuffles, and four lanes hold two 32-dim q8 blocks (r is a multiple of 64). A group
// of lanes takes `per` heads of its row, so that with many rows the angles are made once
// for several heads. Each thread reads its 16 values before it writes them: out may
// be q.
#include <cmath>

#include <cuda_runtime.h>

#include "ops_internal.cuh"
#include "q8_codec.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kBlock = 256;

struct RopeArgs {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_dense q, out, k, v;
  mk_rope rope;
  const int32_t* parents;
  const int32_t* positions;
  int hq, heads, per;       // heads: of q, k and v; per: heads of a group
  uint32_t row_groups;      // groups per row
  int lanes_log2, row0, n;  // lanes of a group; rows [row0, row0 + n) of this launch
};

template <int DT, bool Q8, bool VEC>
__global__ void __launch_bounds__(kBlock) rope_write_kernel(const __grid_constant__ RopeArgs a) {
  using T = typename Elem<DT>::T;
  const int lanes = 1 << a.lanes_log2, c = threadIdx.x & (lanes - 1);
  const uint32_t group = blockIdx.x * (kBlock >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
  const uint32_t g = group / a.row_groups;
  const int part = group - g * a.row_groups;
  const bool live = g < static_cast<uint32_t>(a.n);
  const int row = a.row0 + (live ? static_cast<int>(g) : a.n - 1);  // groups behind the end shadow the last row
  const int lane = threadIdx.x & 31;
  const uint32_t mask = ((1u << lanes) - 1) << (lane & ~(lanes - 1));
  const int dh = a.pool.dh, rot = a.rope.rot, hkv = a.pool.hkv;
  // the lane's dims: eight from lo, eight from lo + step
  const bool in = c < dh / 16;  // (head dim 192 leaves four lanes of sixteen idle)
  const int ci = in ? c : 0, turned = rot / 16;
  const bool turns = ci < turned;
  const int lo = turns ? 8 * ci : rot + 8 * (ci - turned), step = turns ? rot / 2 : (dh - rot) / 2;

  int token = -1, pos = 0, seq = -1;
  float cs[8], sn[8];
  bool looked = false, angles = false;
  for (int it = 0; it < a.per; ++it) {
    const int slot = part + it * static_cast<int>(a.row_groups);
    const bool has = slot < a.heads;
    const int h = has ? slot : a.heads - 1;
    const int kind = h < a.hq ? 0 : h < a.hq + hkv ? 1 : 2, head = kind == 0 ? h : kind == 1 ? h - a.hq : h - a.hq - hkv;
    const mk_dense& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const T* p = static_cast<const T*>(src.data) + row * src.row_stride + head * src.head_stride + lo;
    float x[8], y[8];
    load8<DT, VEC>(p, x);
    load8<DT, VEC>(p + step, y);
    if (!looked) {  // (behind the first loads: three dependent ones)
      looked = true;
      SeqView v;
      seq = seq_of_row(a.rows, row, v);
      if (seq >= 0) {
        const int node = row - v.r0, at = v.kv_len - v.q_len + node;
        token = token_at(a.rows, a.pool.n_pages, seq, at);
        pos = at;
        if (a.positions) {
          pos = __ldg(a.positions + row);
        } else if (a.parents) {
          pos = at - node;
          for (int n = parent_of(a.parents + v.r0, node); n >= 0; n = parent_of(a.parents + v.r0, n)) ++pos;
        }
      }
    }
    if (kind < 2) {
      if (!angles && turns) {
        angles = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * __ldg(a.rope.turns + lo + i);
          sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31
        }
      }
      const float* gain = kind == 0 ? a.rope.q_gain : a.rope.k_gain;
      if (gain) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
        if (!in) sum = 0.f;
        for (int m = lanes >> 1; m; m >>= 1) sum += __shfl_xor_sync(mask, sum, m);
        const float f = rsqrtf(sum / static_cast<float>(dh) + a.rope.eps);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 gx = __ldg(reinterpret_cast<const float4*>(gain + lo + i));
          const float4 gy = __ldg(reinterpret_cast<const float4*>(gain + lo + step + i));
          x[i] *= f * gx.x; x[i + 1] *= f * gx.y; x[i + 2] *= f * gx.z; x[i + 3] *= f * gx.w;
          y[i] *= f * gy.x; y[i + 1] *= f * gy.y; y[i + 2] *= f * gy.z; y[i + 3] *= f * gy.w;
        }
      }
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = x[i] * cs[i] - y[i] * sn[i];
          y[i] = y[i] * cs[i] + x[i] * sn[i];
          x[i] = z;
        }
      }
    }
    if (kind == 0) {
      if (live && has && in && seq >= 0) {
        T* o = static_cast<T*>(a.out.data) + row * a.out.row_stride + head * a.out.head_stride + lo;
        store8<DT, VEC>(o, x);
        store8<DT, VEC>(o + step, y);
      }
      continue;
    }
    const bool store = live && has && in && token >= 0;
    const int64_t e = ((static_cast<int64_t>(token / kPage) * hkv + head) * kPage + token % kPage) * dh + lo;
    void* pool = kind == 1 ? a.pool.k : a.pool.v;
    if constexpr (!Q8) {
      if (store) {
        store8<MK_F16, true>(static_cast<__half*>(pool) + e, x);
        store8<MK_F16, true>(static_cast<__half*>(pool) + e + step, y);
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float* z = half ? y : x;
        float m = fabsf(z[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(z[j]));
        m = fmaxf(m, __shfl_xor_sync(mask, m, 1));  // four lanes hold a block of 32
        m = fmaxf(m, __shfl_xor_sync(mask, m, 2));
        const float d = q8_scale(m);
        uint32_t w[2];
        q8_codes<8>(z, d, m, w);
        if (store) {
          const int64_t at = e + half * step;
          *reinterpret_cast<uint2*>(static_cast<int8_t*>(pool) + at) = make_uint2(w[0], w[1]);
          if ((c & 3) == 0) static_cast<__half*>(kind == 1 ? a.pool.k_scale : a.pool.v_scale)[at / 32] = __float2half_rn(d);
        }
      }
    }
  }
}

using Kernel = void (*)(const RopeArgs);
template <int DT>
Kernel pick(bool q8, bool vec) {
  return q8 ? (vec ? rope_write_kernel<DT, true, true> : rope_write_kernel<DT, true, false>)
            : (vec ? rope_write_kernel<DT, false, true> : rope_write_kernel<DT, false, false>);
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_rope_turns(int32_t rot, double base, const double* freq, uint64_t* turns) {
  if (rot < 0 || rot % 2 || rot > 65536 || (rot && !turns) || (!freq && !(base > 0.0 && std::isfinite(base)))) return MK_ERR_INVALID;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = freq ? freq[i] : std::pow(base, -2.0 * i / rot);
    if (!std::isfinite(f)) return MK_ERR_INVALID;
    double t = std::fmod(f / 6.283185307179586476925, 1.0);
    if (t < 0.0) t += 1.0;
    const double x = std::ldexp(t, 64);
    turns[i] = x < 18446744073709551616.0 ? static_cast<uint64_t>(x) : 0;
  }
  return MK_OK;
}

extern "C" mk_status mk_rope_write(const mk_kv_pool* pool, const mk_kv_rows* rows, const mk_rope_args* r, void* stream) {
  using namespace mk::ops;
  mk_status st = check_pool(pool);
  if (st == MK_OK) st = check_rows(rows);
  if (st != MK_OK) return st;
  if (!r || r->dtype < MK_F32 || r->dtype > MK_BF16 || r->hq <= 0) return MK_ERR_INVALID;
  const mk_rope& p = r->rope;
  if (p.rot < 0 || p.rot > pool->dh || !(p.eps >= 0.f) || !std::isfinite(p.eps) || (r->parents && r->positions)) return MK_ERR_INVALID;
  if (p.rot % 64) return MK_ERR_UNSUPPORTED;
  if (p.rot && (!p.turns || reinterpret_cast<uintptr_t>(p.turns) & 7u)) return MK_ERR_INVALID;
  if (!aligned16(p.q_gain) || !aligned16(p.k_gain)) return MK_ERR_INVALID;
  if (rows->n_seqs == 0 || rows->n_rows == 0) return MK_OK;
  const uintptr_t low = elem_bytes(r->dtype) - 1;
  for (const mk_dense* d : {&r->q, &r->out, &r->k, &r->v})
    if (!d->data || (reinterpret_cast<uintptr_t>(d->data) & low)) return MK_ERR_INVALID;
  const int64_t heads = static_cast<int64_t>(r->hq) + 2ll * pool->hkv;
  if (heads > (1 << 20)) return MK_ERR_UNSUPPORTED;
  const bool vec = dense_vec(r->q, r->dtype) && dense_vec(r->out, r->dtype) && dense_vec(r->k, r->dtype) && dense_vec(r->v, r->dtype);
  const bool q8 = pool->kv_dtype == MK_KV_Q8;
  const Kernel fn = r->dtype == MK_F32 ? pick<MK_F32>(q8, vec) : r->dtype == MK_F16 ? pick<MK_F16>(q8, vec) : pick<MK_BF16>(q8, vec);
  RopeArgs a{*pool, *rows, r->q, r->out, r->k, r->v, p, r->parents, r->positions, r->hq, static_cast<int>(heads), 1, 0, 0, 0, 0};
  a.lanes_log2 = pool->dh == 64 ? 2 : pool->dh == 128 ? 3 : 4;
  const int groups = kBlock >> a.lanes_log2;  // of a block
  // One head a group while that is no more than four blocks an SM; with more rows four heads.
  a.per = rows->n_rows * heads <= 600ll * groups ? 1 : 4;
  a.row_groups = static_cast<uint32_t>((heads + a.per - 1) / a.per);
  const int64_t slab = (1ll << 30) / (a.row_groups << a.lanes_log2);  // threads of one launch stay below 2^31
  for (int64_t r0 = 0; r0 < rows->n_rows; r0 += slab) {
    a.row0 = static_cast<int>(r0);
    a.n = static_cast<int>(rows->n_rows - r0 < slab ? rows->n_rows - r0 : slab);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.n) * a.row_groups + groups - 1) / groups));
    cfg.blockDim = dim3(kBlock);
    cfg.stream = static_cast<cudaStream_t>(stream);
    if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
  }
  return MK_OK;
}
