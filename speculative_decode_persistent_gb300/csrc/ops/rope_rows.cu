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
// shuffles, and four lanes hold two 32-dim q8 blocks (r is a multiple of 64). Such a
// group of lanes takes one head, whose gains stay in registers, of PER rows at a time and
// reads the next ones ahead. The block's threads look all of its rows up and make their
// sines and cosines once for all heads, in shared memory; with many rows there are as many
// blocks as are resident, so that this is paid once. Each thread reads its 16 values of a
// head before it writes them: out may be q.
//
// Bound and measured. Many rows: 8,192 rows of 24 + 4 + 4 heads of 256 (bf16, 268 MB) in 49 us,
// 5.4 TB/s; ncu has 57 % of the issue slots busy and 16 warps an SM, which wait on their own
// arithmetic and on shared memory. The same into a q8 pool takes 80 us (3.1 TB/s; the codec's
// instructions on top: 51 % of the issue slots, DRAM at 34 %), in fp32 100 us into an fp16 pool and
// 99 into a q8 one (5.0 and 4.9 TB/s). Few rows: the launch and three dependent loads of the lookup
// (64 rows into a q8 pool with their reading back, two calls: 12 to 13 us).
#include <cmath>
#include <type_traits>

#include <cuda_runtime.h>

#include "ops_internal.cuh"
#include "q8_codec.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kBlock = 256;
// Rows of a group at a time, where there are many. (8,192 rows of 32 heads of 256, bf16, four rows and two blocks an SM: 52 us; two
// and three: 56; two and four, nothing read ahead: 62; one and six: 74. What is on its way counts.)
constexpr int kPer = 4, kPerF32 = 2;
constexpr int kMaxRows = 256;  // of a block
constexpr int kTable = 40960;  // bytes of its sines and cosines, at most (84 rows of 64 dims take 22 KB)

struct RopeArgs {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_dense q, out, k, v;
  mk_rope rope;
  const int32_t* parents;
  const int32_t* positions;
  int hq, heads;                                       // heads of q; of q, k and v
  int block_heads, head_blocks, group_rows, batches;   // a block's heads; blocks per rows; groups per head; times PER rows
  int lanes_log2, row0, n;         // lanes of a group; rows [row0, row0 + n) of this launch
  float inv_dh;
};

// Eight values as loaded.
template <int DT>
struct Raw {
  uint4 w[DT == MK_F32 ? 2 : 1];
};
template <int DT, bool VEC>
__device__ __forceinline__ Raw<DT> fetch8(const typename Elem<DT>::T* p) {
  Raw<DT> r;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    alignas(16) typename Elem<DT>::T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[i];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) r.w[i] = reinterpret_cast<const uint4*>(t)[i];
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void values8(const Raw<DT>& r, float* x) {
  const typename Elem<DT>::T* t = reinterpret_cast<const typename Elem<DT>::T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::get(t[i]);
}

// Eight values rounded and stored, two a conversion.
template <int DT, bool VEC>
__device__ __forceinline__ void put8(typename Elem<DT>::T* p, const float* x) {
  if constexpr (DT == MK_F32 || !VEC) {
    store8<DT, VEC>(p, x);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = DT == MK_F16 ? pack_half2(x[2 * i], x[2 * i + 1]) : pack_bf162(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A head's (mean x^2 + eps)^-1/2 where the squares leave 32 bits, in two factors (their product may leave them too): the
// power of two that brings the largest value to [1, 4), and the rest. 1 and `plain` where there is no such power (0, infinite,
// NaN), and where eps is so far above the squares that it leaves 32 bits with them: then `plain` is eps's alone.
__device__ __forceinline__ float2 norm_factors(const float (&x)[8], const float (&y)[8], bool in, int lanes, uint32_t mask, float inv_dh, float eps,
                                               float plain) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
    if (x[i] != x[i] || y[i] != y[i]) top = INFINITY;
  }
  if (!in) top = 0.f;
  for (int m = lanes >> 1; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, m));
  if (!(top > 0.f && top < INFINITY)) return make_float2(1.f, plain);
  // 2^-e with 2^e near top, kept normal, as is its reciprocal
  const float s = __uint_as_float(static_cast<uint32_t>(254 - min(max(static_cast<int>(__float_as_uint(top) >> 23), 1), 253)) << 23);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += (x[i] * s) * (x[i] * s) + (y[i] * s) * (y[i] * s);
  if (!in) sum = 0.f;
  for (int m = lanes >> 1; m; m >>= 1) sum += __shfl_xor_sync(mask, sum, m);
  const float e = eps * s * s;
  return e < INFINITY ? make_float2(s, rsqrtf(fmaf(sum, inv_dh, e))) : make_float2(1.f, plain);
}

template <int DT, bool Q8, bool VEC, int PER>
__global__ void __launch_bounds__(kBlock, 2) rope_write_kernel(const __grid_constant__ RopeArgs a) {
  using T = typename Elem<DT>::T;
  wait_for_previous();
  __shared__ int row_token[kMaxRows], row_pos[kMaxRows];  // token: -2 for rows of no sequence
  extern __shared__ __align__(16) float table[];          // [rows of the block][2][rot / 2]: cosines, sines
  const int tid = threadIdx.x, lanes = 1 << a.lanes_log2, c = tid & (lanes - 1), group = tid >> a.lanes_log2;
  const int rb = static_cast<int>(blockIdx.x) / a.head_blocks, h0 = (static_cast<int>(blockIdx.x) - rb * a.head_blocks) * a.block_heads;
  const int r0 = rb * a.batches * a.group_rows * PER;  // the block's first row, of this launch
  const int n_rows = min(a.batches * a.group_rows * PER, a.n - r0);
  const int lane = tid & 31;
  const uint32_t mask = ((1u << lanes) - 1) << (lane & ~(lanes - 1));
  const int dh = a.pool.dh, rot = a.rope.rot, half = rot / 2, hkv = a.pool.hkv;
  // the lane's dims: eight from lo, eight from lo + step
  const bool in = c < dh / 16;  // (head dim 192 leaves four lanes of sixteen idle)
  const int ci = in ? c : 0, turned = rot / 16;
  const bool turns = ci < turned;
  const int lo = turns ? 8 * ci : rot + 8 * (ci - turned), step = turns ? half : (dh - rot) / 2;

  // the group's head and first row (the others lie group_rows apart); groups behind the last head have none
  const int row_lane = group / a.block_heads, g = h0 + group - row_lane * a.block_heads;
  const int first = row_lane < a.group_rows && g < a.heads ? row_lane : n_rows;
  const int kind = g < a.hq ? 0 : g < a.hq + hkv ? 1 : 2;  // q, k, v
  const int head = kind == 0 ? g : kind == 1 ? g - a.hq : g - a.hq - hkv;
  const mk_dense& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const T* p = static_cast<const T*>(src.data) + (a.row0 + r0 + first) * src.row_stride + head * src.head_stride + lo;
  const int64_t next = a.group_rows * src.row_stride;
  struct Batch {
    Raw<DT> x[PER], y[PER];
  };
  auto fetch = [&](int row) {  // of the group's next rows, from `row` on
    Batch t;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      if (row + u * a.group_rows >= n_rows) break;
      t.x[u] = fetch8<DT, VEC>(p);
      t.y[u] = fetch8<DT, VEC>(p + step);
      p += next;
    }
    return t;
  };
  Batch now = fetch(first);
  for (int i = tid; i < n_rows; i += kBlock) {
    const int row = a.row0 + r0 + i;
    SeqView v;
    const int seq = seq_of_row(a.rows, row, v);
    int token = -2, pos = 0;
    if (seq >= 0) {
      const int node = row - v.r0, at = v.kv_len - v.q_len + node;
      token = token_at(a.rows, a.pool.n_pages, seq, at);
      pos = at;
      if (a.positions) {
        pos = a.positions[row];
      } else if (a.parents) {
        pos = at - node;
        for (int n = parent_of(a.parents + v.r0, node); n >= 0; n = parent_of(a.parents + v.r0, n)) ++pos;
      }
    }
    row_token[i] = token;
    row_pos[i] = pos;
  }
  __syncthreads();
  if (h0 < a.hq + hkv) {  // (a block of v alone turns nothing)
    for (int i = tid; i < n_rows * half; i += kBlock) {
      const int r = i / half, j = i - r * half;
      const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(row_pos[r])) * a.rope.turns[j];
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
      table[r * rot + j] = cs;
      table[r * rot + half + j] = sn;
    }
  }
  const float* const gain = kind == 0 ? a.rope.q_gain : kind == 1 ? a.rope.k_gain : nullptr;
  uint64_t gx[4], gy[4];
  if (gain) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const ulonglong2 g0 = *reinterpret_cast<const ulonglong2*>(gain + lo + 2 * i);
      const ulonglong2 g1 = *reinterpret_cast<const ulonglong2*>(gain + lo + step + 2 * i);
      gx[i] = g0.x; gx[i + 1] = g0.y;
      gy[i] = g1.x; gy[i + 1] = g1.y;
    }
  }
  __syncthreads();
  T* const out = static_cast<T*>(a.out.data) + (a.row0 + r0) * a.out.row_stride + head * a.out.head_stride + lo;
  // One head of one row. A head whose squares leave 32 bits is left (true) by the first call, and taken with `rare` set.
  auto turn = [&](const Raw<DT>& rx, const Raw<DT>& ry, int row, auto rare) {
    const int token = row_token[row];
    float x[8], y[8];
    values8<DT>(rx, x);
    values8<DT>(ry, y);
    if (kind < 2) {
      // two values an instruction
      uint64_t x2[4], y2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x2[i] = pack2(x[2 * i], x[2 * i + 1]);
        y2[i] = pack2(y[2 * i], y[2 * i + 1]);
      }
      if (gain) {
        uint64_t s2 = mul2(x2[0], x2[0]), s3 = mul2(y2[0], y2[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s2 = fma2(x2[i], x2[i], s2);
          s3 = fma2(y2[i], y2[i], s3);
        }
        float s0, s1;
        unpack2(add2(s2, s3), s0, s1);
        float sum = in ? s0 + s1 : 0.f;
        sum += __shfl_xor_sync(mask, sum, 1);
        sum += __shfl_xor_sync(mask, sum, 2);
        if (lanes > 4) sum += __shfl_xor_sync(mask, sum, 4);
        if (lanes > 8) sum += __shfl_xor_sync(mask, sum, 8);
        float f = rsqrtf(fmaf(sum, a.inv_dh, a.rope.eps));
        if constexpr (decltype(rare)::value) {
          const float2 sf = norm_factors(x, y, in, lanes, mask, a.inv_dh, a.rope.eps, f);
          const uint64_t p2 = pack2(sf.x, sf.x);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x2[i] = mul2(x2[i], p2);
            y2[i] = mul2(y2[i], p2);
          }
          f = sf.y;
        } else if (DT != MK_F16 && (!(sum < 3e38f) || (sum < 1e-30f && a.rope.eps < 1e-30f))) {  // (binary16's squares fit)
          return true;
        }
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x2[i] = mul2(mul2(x2[i], f2), gx[i]);  // (x f is at most dh^1/2; f g may leave 32 bits)
          y2[i] = mul2(mul2(y2[i], f2), gy[i]);
        }
      }
      if (turns) {
        const float* cs = table + row * rot + lo;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(cs + 2 * i);
          const float4 s4 = *reinterpret_cast<const float4*>(cs + half + 2 * i);
          const uint64_t sn[2] = {pack2(s4.x, s4.y), pack2(s4.z, s4.w)}, neg[2] = {pack2(-s4.x, -s4.y), pack2(-s4.z, -s4.w)};
          const uint64_t cc[2] = {c2.x, c2.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint64_t z = fma2(x2[i + j], cc[j], mul2(y2[i + j], neg[j]));
            y2[i + j] = fma2(y2[i + j], cc[j], mul2(x2[i + j], sn[j]));
            x2[i + j] = z;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unpack2(x2[i], x[2 * i], x[2 * i + 1]);
        unpack2(y2[i], y[2 * i], y[2 * i + 1]);
      }
    }
    if (kind == 0) {
      if (in && token != -2) {
        T* o = out + row * a.out.row_stride;
        put8<DT, VEC>(o, x);
        put8<DT, VEC>(o + step, y);
      }
      return false;
    }
    const bool store = in && token >= 0;
    const int64_t e = ((static_cast<int64_t>(token / kPage) * hkv + head) * kPage + token % kPage) * dh + lo;
    void* pool = kind == 1 ? a.pool.k : a.pool.v;
    if constexpr (!Q8) {
      if (store) {
        put8<MK_F16, true>(static_cast<__half*>(pool) + e, x);
        put8<MK_F16, true>(static_cast<__half*>(pool) + e + step, y);
      }
    } else {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const float* z = side ? y : x;
        float m = fabsf(z[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(z[j]));
        m = fmaxf(m, __shfl_xor_sync(mask, m, 1));  // four lanes hold a block of 32
        m = fmaxf(m, __shfl_xor_sync(mask, m, 2));
        const float d = q8_scale(m);
        uint32_t w[2];
        q8_codes<8>(z, d, m, w);
        if (store) {
          const int64_t at = e + side * step;
          *reinterpret_cast<uint2*>(static_cast<int8_t*>(pool) + at) = make_uint2(w[0], w[1]);
          if ((c & 3) == 0) static_cast<__half*>(kind == 1 ? a.pool.k_scale : a.pool.v_scale)[at / 32] = __float2half_rn(d);
        }
      }
    }
    return false;
  };
  uint64_t left = 0;  // the group's rows that were, by their number
  for (int row = first, i = 0; row < n_rows; row += PER * a.group_rows, i += PER) {  // (whole groups)
    Batch then;
    if (PER > 1 && row + PER * a.group_rows < n_rows) then = fetch(row + PER * a.group_rows);
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (row + u * a.group_rows < n_rows && turn(now.x[u], now.y[u], row + u * a.group_rows, std::false_type())) left |= 1ull << (i + u);
    if (PER > 1) now = then;
  }
  for (; left; left &= left - 1) {
    const int row = first + (__ffsll(static_cast<long long>(left)) - 1) * a.group_rows;
    const T* q = static_cast<const T*>(src.data) + (a.row0 + r0 + row) * src.row_stride + head * src.head_stride + lo;
    turn(fetch8<DT, VEC>(q), fetch8<DT, VEC>(q + step), row, std::true_type());
  }
}

using Kernel = void (*)(const RopeArgs);
template <int DT, int PER>
Kernel pick(bool q8, bool vec) {
  return q8 ? (vec ? rope_write_kernel<DT, true, true, PER> : rope_write_kernel<DT, true, false, PER>)
            : (vec ? rope_write_kernel<DT, false, true, PER> : rope_write_kernel<DT, false, false, PER>);
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
  RopeArgs a{*pool, *rows, r->q, r->out, r->k, r->v, p, r->parents, r->positions, r->hq, static_cast<int>(heads), 1, 1, 1, 1, 0, 0, 0, 1.f / static_cast<float>(pool->dh)};
  a.lanes_log2 = pool->dh == 64 ? 2 : pool->dh == 128 ? 3 : 4;
  const int groups = kBlock >> a.lanes_log2;  // of a block
  // A row a group while that makes no more than 400 blocks (32 heads of 256: 152 rows 4.2 against 6.2 us, 256 rows 7.2
  // against 6.6, 400 rows 7.6 against 6.2).
  const bool many = rows->n_rows * heads > 400ll * groups;
  a.head_blocks = static_cast<int>((heads + groups - 1) / groups);
  a.block_heads = static_cast<int>((heads + a.head_blocks - 1) / a.head_blocks);
  a.group_rows = groups / a.block_heads;
  int block_rows = a.group_rows * (!many ? 1 : r->dtype == MK_F32 ? kPerF32 : kPer);
  if (many) {  // as many batches a block as leave 304 blocks, two an SM, or, where shared memory ends before, a few times as many
    const int64_t blocks = (rows->n_rows + block_rows - 1) / block_rows * a.head_blocks;
    const int fit = kTable / 4 / (p.rot > 64 ? p.rot : 64), room = fit < kMaxRows ? fit : kMaxRows, rows_most = 64 * a.group_rows;
    const int most = (room < rows_most ? room : rows_most) / block_rows;  // (64 rows a group: they are numbered in 64 bits)
    const int64_t waves = (blocks + 304ll * most - 1) / (304ll * most);
    a.batches = static_cast<int>((blocks + 304 * waves - 1) / (304 * waves));
    block_rows *= a.batches;
  }
  const Kernel fn = many ? (r->dtype == MK_F32 ? pick<MK_F32, kPerF32>(q8, vec) : r->dtype == MK_F16 ? pick<MK_F16, kPer>(q8, vec) : pick<MK_BF16, kPer>(q8, vec))
                         : (r->dtype == MK_F32 ? pick<MK_F32, 1>(q8, vec) : r->dtype == MK_F16 ? pick<MK_F16, 1>(q8, vec) : pick<MK_BF16, 1>(q8, vec));
  const int64_t slab = (1ll << 30) / a.head_blocks / block_rows * block_rows;  // blocks of one launch stay below 2^31
  for (int64_t r0 = 0; r0 < rows->n_rows; r0 += slab) {
    a.row0 = static_cast<int>(r0);
    a.n = static_cast<int>(rows->n_rows - r0 < slab ? rows->n_rows - r0 : slab);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>((a.n + block_rows - 1) / block_rows) * a.head_blocks));
    if (launch_early(fn, grid, dim3(kBlock), sizeof(float) * block_rows * p.rot, static_cast<cudaStream_t>(stream), a) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
  }
  return MK_OK;
}
