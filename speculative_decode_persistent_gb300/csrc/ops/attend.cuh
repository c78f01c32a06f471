// Attention of a chunk of new rows over the paged cache, on the tensor cores.
//
// Mathematics. For a row at position p: s_t = scale q.k_t over the tokens it
// sees, out = sum_t 2^(s_t' - m) v_t / sum_t 2^(s_t' - m) with s' = s log2(e)
// and m any reference near the maximum: one pass over the tokens, 128 at a
// time. m moves only when a score passes it by more than kLazy, so the output
// accumulator is rescaled a few times per row, not once per block of tokens. The
// weights are 2^kLift times that (it cancels): their binary16 values then reach
// from 2^15 down to 2^-24, so what the product drops of a weight is below
// 2^-(25 + kLift) of the row's largest.
//
// Shape. The (row, query head) pairs that share a kv head are the rows of a
// tile, 128 of them per thread block (row R of a sequence is token R / group,
// head R % group of the kv head's group). S = Q K^T [128 x 128] and O += P V
// [128 x dh] run as tcgen05.mma with S (two buffers), P (binary16, over S's
// own columns) and O in tensor memory: 2 x 128 + 256 of its 512 columns. P is
// the A operand straight from tensor memory; K is the K-major and V the
// MN-major B operand as TMA lays the pages down (128-byte swizzle).
//
// CG = 1: a block works alone. CG = 2: two blocks of a cluster share one tile
// of 256 rows; each holds half of every K and V block and the instruction
// reads both halves, so a block fetches and stores half the bytes per product.
//
// Work. All (sequence, kv head, tile) items are cut into 128-token blocks of
// what their rows can see (a window skips the middle). The blocks of all items,
// each item's behind a few units that stand for its start and end (query
// rows, result), form one line that is cut evenly among the workers (blocks or
// pairs). An item cut in two or more leaves unnormalised parts, which
// attend_join adds in a fixed order: results do not depend on timing. Every
// worker finds its piece from the lengths on the device, so nothing is planned
// on the host.
//
// Operand units in shared memory, 128-byte rows of 64 dims (a slab), swizzled:
// K as [8 tokens][slab][8 rows], V as [page][slab][16 rows], so that one copy
// brings all slabs of its tokens and a product of 16 tokens reads one page.
//
// Warps: 0-7 take the softmax and write results (two threads a row, 64 tokens
// each, so that a block's softmax is shorter than its products), 8 copies
// pages, 9 issues products, 10-15 prepare operands: they load Q, turn q8 codes
// into binary16 tiles, and clear what must not enter a product (below).
//
// Unseen values. A masked score is replaced before the softmax, so K may hold
// anything. A masked probability is 0, but 0 x inf is NaN inside a product:
// in blocks that some row sees only in part, non-finite V values are cleared
// in shared memory before the product, and rows that do see one add it when
// they write their result (a rare path). Missing pages arrive as zeros.
//
// Large q8 values. A q8 block holds up to 127 x 65504, its operands are binary16.
// The softmax warps note the first segment with a scale of 512 or more; from it
// on a worker writes no result, and takes its segments again with code that lets
// the values of such tokens enter the products as 2^-8 of themselves. There the
// preparing and the softmax warps find the tokens by their scales, each for itself:
// the factor of a K token goes into its scores, that of a V token into its weight's
// exponent (also in the running maximum, so that the weight stays a binary16
// number) and out of the sum of the weights. (That code in the only pass: 69 -> 83 us
// for 4 x 3 rows over 23K tokens, 202 -> 252 us for 512 rows over 20K. Two passes take
// 2.7 times as long as one: 204 and 556 us.)
//
// Bound and measured (24 query heads, 4 kv heads of 256). Many rows: the
// products; 2,048 rows over 20,512 fp16 tokens in 559 us, 1,755 TFLOP/s, over
// q8 tokens in 682 us, where converting the codes takes as long. Few rows: the
// pages; 4 x 3 rows over 23,003 fp16 tokens each in 71 us, 5.3 TB/s, q8 in 71 us
// (200 MB; converting again). One row over 4,097 tokens: 15.8 us, latency.
//
// Every wait is bounded; a worker that gives up writes NaN for its rows. Before its
// blocks end it waits (with a limit again) for the copies and products that are
// still under way: they would reach shared and tensor memory of the next blocks.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <type_traits>

#include "ops_internal.cuh"
#include "sm103.cuh"

namespace mk {
namespace ops {

constexpr int kBN = 128;             // tokens per block: eight pages
constexpr int kMaxWorkers = 160;     // at least the SM count
// Reference of the softmax (see above), as powers of two: how far a score may pass
// it, and what the weights are raised by. (4 and 11 against 8 and 7: 2^4 times finer
// weights; the same times, but 2 % more where a window begins with a few sinks.)
constexpr float kLazy = 4.f, kLift = 15.f - kLazy;
constexpr int kJoinSplit = 8;        // join blocks per cut
// An item's start and end in blocks, 4 for one block, 8 for a pair (a 4,096-row
// prompt over 24 heads of 256: 2 208 us, 4 178 us, 8 166 us; one row over 4K q8
// tokens in one block: 4 17.2 us, 8 18.2 us).
__host__ __device__ constexpr int item_cost(int m) { return m / 32; }

// A worker's first item, when it began at an earlier worker: what the join needs.
struct JoinInfo {
  int r0, h, mt, w0, w1, slot0, rows, pad;  // w0 < 0: nothing to join here; r0: the sequence's first row
};

struct AttendParams {
  mk_kv_pool pool;
  mk_kv_rows rows;
  mk_dense q, gate, out;
  int hq, G, g_inv, dtype, window, sinks, workers;  // g_inv = 2^20 / G + 1: x / G = x g_inv >> 20 for x < 2^20 / G
  float c;         // scale x log2(e)
  int vq, vo, vg;  // 16-byte access to q, out, gate (out: 2 with 32 bytes)
  int skip;        // test hook: the worker whose queries are not handed over, -1: none
  int wait_us;     // after which a wait gives up
  JoinInfo* join;  // [kMaxWorkers]
  float2* ml;      // [2 workers][128 CG] reference and sum of a part
  float* part;     // [2 workers][128 CG][dh] unnormalised output
};

// ------------------------------------------------------------------ geometry
// Tile mt of a sequence: M rows of (token, head in group) pairs.
struct Tile {
  int rows;         // valid rows
  int t0, h0;       // token (within the new rows) and head (within the group) of the first row
  int p0, p1;       // positions of its first and last token
  int nblk;         // 128-token blocks some row may see, at least 1
  int sink_b, lo;   // block i is i < sink_b ? i : lo + i - sink_b
  __device__ __forceinline__ int block(int i) const { return i < sink_b ? i : lo + i - sink_b; }
};
__device__ __forceinline__ int tiles_of(const SeqView& v, int G, int M) { return (v.q_len * G + M - 1) / M; }
__device__ __forceinline__ Tile make_tile(const SeqView& v, int G, int M, int mt, int window, int sinks) {
  Tile t;
  const int R0 = mt * M, R1 = min(R0 + M, v.q_len * G);
  t.rows = R1 - R0;
  t.t0 = R0 / G;
  t.h0 = R0 - t.t0 * G;
  t.p0 = v.kv_len - v.q_len + t.t0;
  t.p1 = v.kv_len - v.q_len + (R1 - 1) / G;
  t.sink_b = t.lo = 0;
  t.nblk = 1;
  if (t.p1 >= 0) {
    const int hi = t.p1 / kBN;
    if (window > 0) {
      t.lo = max(0, t.p0 - window + 1) / kBN;
      t.sink_b = (min(sinks, t.p1 + 1) + kBN - 1) / kBN;
      if (t.sink_b >= t.lo) t.lo = t.sink_b = 0;
    }
    t.nblk = t.sink_b + hi - t.lo + 1;
  }
  return t;
}
// Token and head of row r (below 256) of a tile, relative to its first row's token.
struct RowOf {
  int tok, head;
};
__device__ __forceinline__ RowOf row_of(const Tile& t, int r, int G, int g_inv) {
  const int x = t.h0 + r, q = (x * g_inv) >> 20;
  return {t.t0 + q, x - q * G};
}
// Whether rows at positions p0..p1 all see every token of block b.
__device__ __forceinline__ bool block_full(int b, int p0, int p1, int window, int sinks) {
  const int last = b * kBN + kBN - 1;
  return last <= p0 && (window == 0 || b * kBN > p1 - window || last < sinks);
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// Tokens base .. base+31 that a row at position p sees (missing pages aside).
__device__ __forceinline__ uint32_t seen_bits(int p, int base, int window, int sinks) {
  uint32_t m = low_bits(p - base + 1);
  if (window > 0) m &= ~low_bits(p - window + 1 - base) | low_bits(sinks - base);
  return m;
}

// A q8 token is large when one of its 2 NS scales is 512 or more (infinite and NaN ones too): 128 times it, the
// largest code, is not a binary16 number. Scales are compared as integers, two at a time, so a sign counts as large.
template <int NS>
__device__ __forceinline__ void token_scales(const uint8_t* scales, uint32_t (&w)[NS]) {
  if constexpr (NS == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(scales);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (NS == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(scales);
    w[0] = x.x; w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) w[i] = reinterpret_cast<const uint32_t*>(scales)[i];
  }
}
template <int N>
__device__ __forceinline__ bool any_large(const uint32_t (&w)[N]) {
  uint32_t top = w[0];
#pragma unroll
  for (int i = 1; i < N; i += 2) top = __vimax3_u16x2(top, w[i], w[i + 1 < N ? i + 1 : i]);
  return max(top >> 16, top & 0xffffu) >= 0x6000u;
}
template <int NS>
__device__ __forceinline__ bool large_token(const uint8_t* scales) {
  uint32_t w[NS];
  token_scales<NS>(scales, w);
  return any_large(w);
}

// Column of S's 128 in which P of token t (even) lies: each half over its own scores.
__host__ __device__ constexpr int p_col(int t) { return t / 64 * 64 + t % 64 / 2; }

// A worker's walk through the line: segments of consecutive blocks of one
// item. Every role walks it for itself.
struct Start {
  int s, h, mt, off, n;  // item, offset into its part of the line, length of the worker's piece
  SeqView v;
};
struct Walk {
  const AttendParams* a;
  int s, h, mt, off, left, n_mt, M, seg;
  SeqView v;
  Tile t;
  int b0, b1;  // block indices [b0, b1) of the current segment
  __device__ __forceinline__ Walk(const AttendParams& p, const Start& st, int M_)
      : a(&p), s(st.s), h(st.h), mt(st.mt), off(st.off), left(st.n), M(M_), seg(-1), v(st.v) {
    n_mt = left > 0 ? tiles_of(v, p.G, M) : 0;
  }
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    if (seg >= 0 && ++mt == n_mt) {
      mt = 0;
      if (++h == a->pool.hkv) {
        h = 0;
        do {
          if (++s >= a->rows.n_seqs) return false;  // (only if the lengths changed under the kernel)
          v = seq_view(a->rows, s);
          n_mt = tiles_of(v, a->G, M);
        } while (n_mt == 0);
      }
    }
    ++seg;
    t = make_tile(v, a->G, M, mt, a->window, a->sinks);
    b0 = max(0, off - item_cost(M));
    b1 = min(t.nblk, max(0, off + left - item_cost(M)));
    left -= t.nblk + item_cost(M) - off;
    off = 0;
    return b1 > b0;  // a piece that ends in an item's start leaves it to the next worker
  }
  __device__ __forceinline__ bool more() const { return left > item_cost(M); }  // another segment follows
  __device__ __forceinline__ bool whole() const { return b0 == 0 && b1 == t.nblk; }
  // Table entry of the block's i-th 16 tokens, -1 behind the table; as loaded,
  // so that a load ahead is waited for only where has_page() looks at it.
  __device__ __forceinline__ int entry(int b, int i) const {
    const int e = b * (kBN / kPage) + i;
    return e < a->rows.table_stride ? __ldg(a->rows.tables + static_cast<int64_t>(s) * a->rows.table_stride + e) : -1;
  }
  __device__ __forceinline__ bool has_page(int entry) const { return entry >= 0 && entry < a->pool.n_pages; }
};

// -------------------------------------------------------------------- layout
// Bytes per row of a q8 tensor-copy box: 128 where every unit's width is a multiple of it.
__host__ __device__ constexpr int q8_box(int ns, int cg) { return ns % 2 || ns / cg == 1 ? 64 : 128; }
template <int NS, bool Q8, int CG>
struct Cfg {
  static constexpr int DH = NS * 64, M = 128 * CG;
  // units: what one ring slot holds, nkeys tokens x nsl slabs of 64 dims
  // K: 64 tokens, all slabs, in pairs that one product reads across two
  // neighbouring slots (kPairK: half the copies); of a q8 pool, whose units
  // should be handed over as soon as they are converted, and of narrow heads
  // all 128 tokens, two slabs each. Of two blocks each has its 64 tokens.
  static constexpr bool kPairK = !Q8 && CG == 1 && NS > 2;
  static constexpr int KU = CG == 2 ? 1 : (NS + 1) / 2;
  static constexpr int VU = CG == 2 ? 1 : NS > 2 ? 2 : 1;  // V: all slabs, split over the tokens (pair: half the slabs)
  static constexpr int kKeysK = CG == 2 || kPairK ? 64 : 128, kKeysV = CG == 2 ? 128 : 128 / VU;
  static constexpr int kSlabsV = CG == 2 ? NS / 2 : NS;
  static __host__ __device__ constexpr int slabs_k(int u) { return CG == 2 || kPairK ? NS : (NS - 2 * u < 2 ? NS - 2 * u : 2); }
  static constexpr int kBoxSlabsK = CG == 2 || kPairK || NS < 2 ? NS : 2;  // slabs a K unit has room for
  static constexpr int kUnitK = kKeysK * kBoxSlabsK * 128, kUnitV = kKeysV * kSlabsV * 128;
  static constexpr int kSlot = kUnitK > kUnitV ? kUnitK : kUnitV;
  static constexpr int kQ = NS * 16384;
  static constexpr int kMisc = 3040;
  static constexpr int kRaw = kSlot / 2 + 128 * NS * 4;  // q8 codes, then 2 NS scales per token
  static constexpr int kBudget = 232448 - kMisc - kQ;
  // binary16 pool: all room for operand units. q8: a block alone keeps two and
  // gives the rest to units as stored, which are what is in flight from memory;
  // a pair, bound by its products, keeps three.
  static constexpr int kFit = kBudget / kSlot;
  static constexpr int kSlots = Q8 ? CG + 1 : kFit > 8 ? 8 : kPairK ? kFit / 2 * 2 : kFit;
  static constexpr int kRawFit = (kBudget - kSlots * kSlot) / kRaw;
  static constexpr int kRawSlots = !Q8 ? 0 : kRawFit > 6 ? 6 : kRawFit;
  static constexpr int kBox = q8_box(NS, CG);
  static constexpr int kSmem = kMisc + kQ + kSlots * kSlot + kRawSlots * kRaw;
  static_assert(!kPairK || (kSlots % 2 == 0 && kSlot == kUnitK && kUnitK == kUnitV), "pairs of K units lie side by side");
  static_assert(kSlots >= 2 && (!Q8 || kRawSlots >= 3) && kSmem <= 232448, "ring");
  static_assert(!Q8 || (slabs_k(0) * 64 % kBox == 0 && kSlabsV * 64 % kBox == 0), "boxes");
};

// 16 warps: 128 registers a thread, which the softmax's 64 live scores need
// (with 20 warps and 96 registers they spilled and the softmax took twice as
// long; ptxas did not use what setmaxnreg would have moved to them).
constexpr int kWarpCopy = 8, kWarpMma = 9, kWarpPrep = 10;
constexpr int kPrep = 6;  // preparing warps
constexpr int kThreads = 32 * (kWarpPrep + kPrep);

// A segment as one softmax warp found it, for all eight: they meet at named
// barriers and must agree on its blocks even if lengths change under the kernel.
struct Segment {
  int s, h, mt, b0, b1, more;
  SeqView v;
  Tile t;
};

struct Misc {
  uint64_t ready[8], full[8], empty[8], raw_full[6], raw_empty[6];
  uint64_t s_full[2], p_ready[2], pv_done, o_full, q_ready, q_free, drained;
  uint32_t tmem;
  int dead[2];  // whether a wait gave up; the microseconds after which one does
  int failed;  // the pair's products stopped before their end: `drained` follows
  Start start;
  int large;             // first segment with large q8 values, INT_MAX: none; the same in both blocks of a pair
  int taken, units, blocks;  // segments, units and blocks of the first pass
  int flag[4];           // segment + 1 in which non-finite V values were cleared
  int raw_pages[6];      // bit i: page i of a raw unit is missing
  Segment segment[2];    // by segment parity
  int8_t qe[3][128];     // per row, by segment modulo 3 (scores run two blocks ahead of their softmax): the power of two its query was divided by
  float swap[2][2][128];  // [block parity][half]: the halves' maxima, at the end their sums
};
static_assert(sizeof(Misc) <= 3040, "misc area");

// Output of eight or more neighbouring dims: gate, rounding, store. Sixteen of
// them go out as one 32-byte sector where the alignment allows: a warp's rows
// lie far apart, and half-filled sectors took twice as long.
template <int N>
__device__ __forceinline__ void put_out(const AttendParams& a, int row, int head, int d0, float* x) {
  const int64_t oo = row * a.out.row_stride + head * a.out.head_stride + d0;
  if (a.gate.data) {
    const int64_t go = row * a.gate.row_stride + head * a.gate.head_stride + d0;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      float g[8];
      if (a.dtype == MK_F16) {
        const __half* gp = static_cast<const __half*>(a.gate.data) + go + i;
        if (a.vg) load8<MK_F16, true>(gp, g); else load8<MK_F16, false>(gp, g);
      } else {
        const __nv_bfloat16* gp = static_cast<const __nv_bfloat16*>(a.gate.data) + go + i;
        if (a.vg) load8<MK_BF16, true>(gp, g); else load8<MK_BF16, false>(gp, g);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i + k] = __fdividef(x[i + k], 1.f + __expf(-g[k]));
    }
  }
  uint16_t* op = static_cast<uint16_t*>(a.out.data) + oo;
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N; i += 2) w[i / 2] = a.dtype == MK_F16 ? pack_half2(x[i], x[i + 1]) : pack_bf162(x[i], x[i + 1]);
  if (N >= 16 && a.vo == 2) {
#pragma unroll
    for (int i = 0; i + 8 <= N / 2; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(op + 2 * i), "r"(w[i]), "r"(w[i + 1]),
                   "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else if (a.vo) {
#pragma unroll
    for (int i = 0; i < N / 2; i += 4) *reinterpret_cast<uint4*>(op + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      op[2 * i] = static_cast<uint16_t>(w[i]);
      op[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// ---------------------------------------------------------------- scheduling
// The line's length and this worker's piece of it. scratch: [n_seqs]. All
// threads of the block call it. (The line has fewer than 2^31 units: the host
// refuses longer ones.)
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  return x;
}
template <int M>
__device__ void find_start(const AttendParams& a, int* scratch, Start* out, int worker, bool leader) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, nw = blockDim.x / 32;
  const int n_seqs = a.rows.n_seqs, hkv = a.pool.hkv;
  // a thread adds up a sequence of few tiles (hundreds of decoding sequences
  // at once), a warp one of many
  constexpr int kFew = 4;
  bool many = false;
  for (int s = threadIdx.x; s < n_seqs; s += blockDim.x) {
    const SeqView v = seq_view(a.rows, s);
    const int n = tiles_of(v, a.G, M);
    int sum = n <= kFew ? 0 : -1;
    for (int mt = 0; mt < min(n, kFew) && sum >= 0; ++mt)
      sum += make_tile(v, a.G, M, mt, a.window, a.sinks).nblk + item_cost(M);
    scratch[s] = sum;
    many |= sum < 0;
  }
  if (__syncthreads_or(many)) {
    for (int s = warp; s < n_seqs; s += nw) {
      if (scratch[s] >= 0) continue;
      const SeqView v = seq_view(a.rows, s);
      const int n = tiles_of(v, a.G, M);
      int sum = 0;
      for (int mt = lane; mt < n; mt += 32) sum += make_tile(v, a.G, M, mt, a.window, a.sinks).nblk + item_cost(M);
      sum = warp_sum(sum);
      __syncwarp();
      if (lane == 0) scratch[s] = sum;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  int total = 0;
  for (int s0 = 0; s0 < n_seqs; s0 += 32) total += warp_sum(s0 + lane < n_seqs ? scratch[s0 + lane] : 0);
  total *= hkv;
  const int quota = max(1, total / a.workers + (total % a.workers > 0));
  const int64_t g = static_cast<int64_t>(worker) * quota;
  const int n = g < total ? min(quota, total - static_cast<int>(g)) : 0, g0 = static_cast<int>(g);
  if (leader && lane == 0) a.join[worker].w0 = -1;
  if (lane == 0) out->n = n;
  if (n <= 0) return;
  // the sequence whose part of the line holds g0, then the head, then the tile
  int at = 0, cost = 0, s = 0;
  for (;; s += 32) {
    if (s >= n_seqs) {  // (only for rows that belong to several sequences, whose sum left 32 bits)
      if (lane == 0) out->n = 0;
      return;
    }
    cost = s + lane < n_seqs ? scratch[s + lane] : 0;
    const int inc = warp_scan(cost * hkv, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, g0 < at + inc);
    if (hit) {
      const int l = __ffs(hit) - 1;
      at += __shfl_sync(0xffffffffu, inc - cost * hkv, l);
      cost = __shfl_sync(0xffffffffu, cost, l);
      s += l;
      break;
    }
    at += __shfl_sync(0xffffffffu, inc, 31);
  }
  const SeqView v = seq_view(a.rows, s);
  const int h = (g0 - at) / cost;
  at += h * cost;
  const int n_mt = tiles_of(v, a.G, M);
  int mt = 0, nblk = 0;
  for (;; mt += 32) {
    if (mt >= n_mt) {  // (only if the lengths changed under the kernel)
      if (lane == 0) out->n = 0;
      return;
    }
    const int nb = mt + lane < n_mt ? make_tile(v, a.G, M, mt + lane, a.window, a.sinks).nblk + item_cost(M) : 0;
    const int inc = warp_scan(nb, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, g0 < at + inc && nb > 0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      at += __shfl_sync(0xffffffffu, inc - nb, l);
      nblk = __shfl_sync(0xffffffffu, nb, l) - item_cost(M);
      mt += l;
      break;
    }
    at += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) {
    *out = Start{s, h, mt, g0 - at, n, v};
    const int first = at + item_cost(M);  // the item's first block
    if (leader && g0 > first) {
      JoinInfo j;
      j.r0 = v.r0;
      j.h = h;
      j.mt = mt;
      j.w0 = first / quota;
      j.w1 = (first + nblk - 1) / quota;
      // the first worker's segment is its first one when its piece begins in this item
      j.slot0 = 2 * j.w0 + (j.w0 * quota >= at ? 0 : 1);
      j.rows = min(M, v.q_len * a.G - mt * M);
      j.pad = 0;
      a.join[worker] = j;
    }
  }
}

// Adds the parts of items that were cut; the cuts' blocks share an item's
// rows. A warp adds a row's parts; where there are fewer rows than blocks
// (decoding over a long cache: many parts) a block's eight warps take the
// parts of one row in turn and add their sums in shared memory (one row over
// 4K tokens: 23.7 -> 16.1 us).
template <int NS, int CG>
__global__ void __launch_bounds__(256) attend_join(const AttendParams a) {
  constexpr int DH = NS * 64, M = 128 * CG, kPer = DH / 32;
  __shared__ float sums[8][DH + 4];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched early: the parts are written from here on
  const JoinInfo j = a.join[blockIdx.x];
  if (j.w0 < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int cuts = j.w1 - j.w0;
  const int share = j.rows <= cuts * static_cast<int>(gridDim.y) ? 8 : 1;  // warps a row: as many as leave no row waiting
  const int first = ((static_cast<int>(blockIdx.x) - j.w0 - 1) * gridDim.y + blockIdx.y) * (8 / share);
  if (first >= j.rows) return;
  for (int r0 = first; r0 < j.rows; r0 += cuts * gridDim.y * (8 / share)) {
    const int r = share == 1 ? r0 + warp : r0;
    if (r < j.rows) {
      float m = -INFINITY;
      for (int k = lane; k <= cuts; k += 32) m = fmaxf(m, a.ml[(k ? 2 * (j.w0 + k) : j.slot0) * M + r].x);
#pragma unroll
      for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      if (m == -INFINITY) m = 0.f;
      float l = 0.f, o[kPer] = {};
#pragma unroll 4
      for (int k = share == 1 ? 0 : warp; k <= cuts; k += share) {
        const int slot = k ? 2 * (j.w0 + k) : j.slot0;
        const float2 x = a.ml[slot * M + r];
        const float f = ex2(x.x - m);
        l += f * x.y;
        const float* p = a.part + (static_cast<int64_t>(slot) * M + r) * DH + lane * kPer;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const float2 y = *reinterpret_cast<const float2*>(p + i);
          o[i] += f * y.x;
          o[i + 1] += f * y.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) sums[warp][lane * kPer + i] = o[i];
      if (lane == 0) sums[warp][DH] = l;
    }
    if (share == 1) __syncwarp(); else __syncthreads();
    // a row's dims, eight per lane
    if (r < j.rows && (share == 1 || warp == 0) && lane < DH / 8) {
      float x[8] = {}, l = 0.f;
      for (int w = 0; w < share; ++w) {
        const float* sum = sums[share == 1 ? warp : w];
        l += sum[DH];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += sum[lane * 8 + i];
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = l == 0.f ? 0.f : x[i] * inv;
      const int R = j.mt * M + r, tok = R / a.G, row = j.r0 + tok, head = j.h * a.G + R - tok * a.G;
      put_out<8>(a, row, head, lane * 8, x);
    }
    if (share == 1) __syncwarp(); else __syncthreads();
  }
}

// The worker's segments, every warp its part. LARGE: once more, from segment `first` on, with large q8 values.
template <int NS, bool Q8, int CG, bool LARGE>
__device__ __forceinline__ void attend_pass(const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv, uint8_t* smem,
                                            uint32_t tm) {
  using C = Cfg<NS, Q8, CG>;
  constexpr int M = C::M, DH = C::DH;
  uint8_t* const sq = smem;                          // Q [NS][128 rows][128 B], swizzled
  uint8_t* const ring = sq + C::kQ;                  // operand units
  uint8_t* const raw = ring + C::kSlots * C::kSlot;  // q8 units as stored
  Misc& ms = *reinterpret_cast<Misc*>(raw + C::kRawSlots * C::kRaw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int rank = CG == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
  const int worker = blockIdx.x / CG;
  volatile int* const dead = ms.dead;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  auto wait1 = [&](uint64_t& b, uint32_t parity) { return bar_wait(smem_u32(&b), parity, dead); };
  auto wait = [&](uint64_t& b, uint32_t parity) { return __all_sync(0xffffffffu, wait1(b, parity)) != 0; };  // whole warps
  // barriers the product-issuing block waits on, reached from both blocks
  auto lead_arrive = [&](uint64_t& b) {
    if (CG == 1) bar_arrive(smem_u32(&b)); else bar_arrive_cluster(peer_addr(smem_u32(&b), 0));
  };

  Walk wk(a, ms.start, M);
  // barriers and buffers go by the number of segments taken so far: seg + shift
  const int first = LARGE ? ms.large : 0, shift = LARGE ? ms.taken - first : 0;
  const int units0 = LARGE ? ms.units : 0, blocks0 = LARGE ? ms.blocks : 0;
  const bool ok0 = !LARGE || !*dead;  // (after a wait that gave up: NaN for the rows that are left)
  auto take = [&] {
    if constexpr (LARGE) {
      while (wk.seg + 1 < first)
        if (!wk.next()) return false;
    }
    return wk.next();
  };

  if (warp == kWarpCopy) {
    // ------------------------------------------------------------ page copies
    int n = units0;  // units issued
    bool ok = ok0;
    // unit u of K (kv = 0) or V of block b, whose page ids the lanes 0..7 hold
    auto unit = [&](auto kvc, auto uc, int pg) {
      constexpr int kv = decltype(kvc)::value, u = decltype(uc)::value;
      constexpr int nkeys = kv ? C::kKeysV : C::kKeysK, np = nkeys / kPage;
      const int p0 = CG == 2 ? (kv ? 0 : 4 * rank) : (kv ? u * C::kKeysV : C::kPairK ? u * 64 : 0) / kPage;
      const int slab0 = CG == 2 ? (kv ? rank * C::kSlabsV : 0) : kv || C::kPairK ? 0 : 2 * u;
      const int none = a.pool.n_pages * a.pool.hkv * kPage;  // a row behind the pool reads as zeros
      // the pages' rows first, then one lane's copies back to back
      int y[np];
#pragma unroll
      for (int i = 0; i < np; ++i) {
        const int page = __shfl_sync(0xffffffffu, pg, (p0 + i) & 7);
        y[i] = wk.has_page(page) ? (page * a.pool.hkv + wk.h) * kPage : none;
      }
      if constexpr (!Q8) {
        // K: boxes of 8 tokens x the unit's slabs (of a page where that is one), V: of a page x the unit's slabs
        const int slot = n % C::kSlots;
        if (!wait(ms.empty[slot], ((n / C::kSlots) & 1) ^ 1)) return false;
        const uint32_t fb = bar(ms.full[slot]), dst = smem_u32(ring + slot * C::kSlot);
        if (elect_one()) {
          constexpr uint32_t kPageBytes = kPage * 128 * (kv ? C::kSlabsV : C::kBoxSlabsK);
          constexpr bool kWhole = kv || C::kBoxSlabsK == 1;  // a page's copy in one
          bar_expect(fb, np * kPageBytes);
#pragma unroll
          for (int i = 0; i < np; ++i) {
            tma_3d(dst + i * kPageBytes, kv ? &tv : &tk, 0, y[i], slab0, fb);
            if (!kWhole) tma_3d(dst + i * kPageBytes + kPageBytes / 2, &tk, 0, y[i] + 8, slab0, fb);
          }
        }
        __syncwarp();
      } else {
        const int slot = n % C::kRawSlots;
        if (!wait(ms.raw_empty[slot], ((n / C::kRawSlots) & 1) ^ 1)) return false;
        const uint32_t gone = __ballot_sync(0xffffffffu, lane < 8 && !wk.has_page(pg));
        const uint32_t mine = (gone >> p0) & ((1u << np) - 1);
        constexpr int kScaleBytes = kPage * NS * 4;
        const uint32_t fb = bar(ms.raw_full[slot]), dst = smem_u32(raw + slot * C::kRaw);
        constexpr int nsl = kv ? C::kSlabsV : C::slabs_k(u), nbx = nsl * 64 / C::kBox;
        if (elect_one()) {
          const uint8_t* scales = static_cast<const uint8_t*>(kv ? a.pool.v_scale : a.pool.k_scale);
          ms.raw_pages[slot] = static_cast<int>(mine);
          bar_expect(fb, nkeys * nsl * 64 + (np - __popc(mine)) * kScaleBytes);
#pragma unroll
          for (int i = 0; i < np; ++i) {
#pragma unroll
            for (int bx = 0; bx < nbx; ++bx)
              tma_2d(dst + (i * nbx + bx) * kPage * C::kBox, kv ? &tv : &tk, slab0 * 64 + bx * C::kBox, y[i], fb);
            if (y[i] != none)
              bulk_copy(dst + C::kSlot / 2 + i * kScaleBytes, scales + static_cast<int64_t>(y[i]) * (NS * 4), kScaleBytes, fb);
          }
        }
        __syncwarp();
      }
      ++n;
      return true;
    };
    auto units = [&](auto kvc, int pg) {
      bool good = unit(kvc, std::integral_constant<int, 0>(), pg);
      if constexpr ((decltype(kvc)::value ? C::VU : C::KU) > 1) good = good && unit(kvc, std::integral_constant<int, 1>(), pg);
      return good;
    };
    while (ok && __any_sync(0xffffffffu, take())) {
      const int b0 = __shfl_sync(0xffffffffu, wk.b0, 0), b1 = __shfl_sync(0xffffffffu, wk.b1, 0);
      int pg = lane < 8 ? wk.entry(wk.t.block(b0), lane) : -1, pg_v = -1;
      for (int i = b0; ok && i <= b1; ++i) {
        const int pg_next = i + 1 < b1 && lane < 8 ? wk.entry(wk.t.block(i + 1), lane) : -1;
        if (i < b1) ok = units(std::integral_constant<int, 0>(), pg);
        if (ok && i > b0) ok = units(std::integral_constant<int, 1>(), pg_v);
        pg_v = pg;
        pg = pg_next;
      }
    }
    {
      // no copy may be in flight when the block goes away (the last units' ones
      // have landed unless a wait gave up): at most one phase per slot is open
      const int ns = Q8 ? C::kRawSlots : C::kSlots;
      for (int k = max(0, n - ns); k < n; ++k) {
        uint64_t& b = Q8 ? ms.raw_full[k % ns] : ms.full[k % ns];
        bar_drain(bar(b), (k / ns) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    // -------------------------------------------------------- product issuer
    // The whole warp walks along, with loop bounds and waits that are uniform
    // by construction (votes, shuffles), and one elected lane issues: so the
    // operands sit in uniform registers. In one lane's own branch each product
    // took about 100 cycles to issue.
    if (rank == 0) {
      constexpr uint32_t kIdS = instr_desc(M, kBN, 0), kIdO = instr_desc(M, DH, 1);
      const uint32_t qa = smem_u32(sq), ra = smem_u32(ring);
      int slot = units0 % C::kSlots, phase = (units0 / C::kSlots) & 1, blk = blocks0;  // ring position, block whose scores come next
      bool ok = ok0;
      auto step_slot = [&] {
        if (++slot == C::kSlots) {
          slot = 0;
          phase ^= 1;
        }
      };
      auto scores = [&]() {  // S[blk & 1] = Q K^T
        const uint32_t d = tm + 256 + (blk & 1) * kBN;
#pragma unroll
        for (int u = 0; u < C::KU; ++u) {
          const int first = slot;
          if (!wait(ms.ready[slot], phase)) return false;
          if (C::kPairK) {
            step_slot();
            if (!wait(ms.ready[slot], phase)) return false;
          }
          tc_fence_after();
          const uint64_t da = smem_desc(qa + (CG == 2 || C::kPairK ? 0 : 2 * u) * 16384, 16, 1024);
          const uint64_t db = smem_desc(ra + first * C::kSlot, 16, C::kBoxSlabsK * 1024);
          if (elect_one()) {
#pragma unroll
            for (int sl = 0; sl < C::slabs_k(u); ++sl)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss<CG>(d, da + sl * 1024 + k * 2, db + sl * 64 + k * 2, kIdS, u + sl + k > 0);
            mma_commit<CG>(bar(ms.empty[first]));
            if (C::kPairK) mma_commit<CG>(bar(ms.empty[slot]));
            if (u + 1 == C::KU || C::kPairK) mma_commit<CG>(bar(ms.s_full[blk & 1]));
          }
          __syncwarp();
          step_slot();
          if (C::kPairK) break;  // (both units at once)
        }
        ++blk;
        return true;
      };
      while (ok && __any_sync(0xffffffffu, take())) {
        const int count = __shfl_sync(0xffffffffu, wk.b1 - wk.b0, 0);
        ok = wait(ms.q_ready, (wk.seg + shift) & 1);
        if (!ok) break;
        tc_fence_after();
        for (int i = 0; i <= count; ++i) {
          if (i < count) {
            ok = scores();
            if (!ok) break;
            if (i + 1 == count) {
              if (elect_one()) mma_commit<CG>(bar(ms.q_free));
              __syncwarp();
            }
          }
          if (i == 0) continue;
          const int pb = blk - (i < count ? 2 : 1);  // the block whose weights are next
          ok = wait(ms.p_ready[pb & 1], (pb >> 1) & 1);
          if (!ok) break;
#pragma unroll
          for (int u = 0; u < C::VU; ++u) {
            ok = wait(ms.ready[slot], phase);
            if (!ok) break;
            tc_fence_after();
            const uint32_t pa = tm + 256 + (pb & 1) * kBN;
            const uint64_t db = smem_desc(ra + slot * C::kSlot, 2048, 1024);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < C::kKeysV / 16; ++k)
                mma_ts<CG>(tm, pa + p_col(u * C::kKeysV + k * 16), db + k * C::kSlabsV * 128, kIdO, u + k > 0 || i > 1);
              mma_commit<CG>(bar(ms.empty[slot]));
              if (u + 1 == C::VU) {
                mma_commit<CG>(bar(ms.pv_done));
                if (i == count) mma_commit<CG>(bar(ms.o_full));
              }
            }
            __syncwarp();
            step_slot();
          }
          if (!ok) break;
        }
      }
      // a wait gave up: what was issued, and its arrivals on both blocks' barriers, come to an end first
      if (ok0 && __any_sync(0xffffffffu, !ok || *dead)) {
        if (elect_one()) {
          for (int k = 0; k < CG; ++k) st_cluster(peer_addr(smem_u32(&ms.failed), k), 1);
          mma_commit<CG>(bar(ms.drained));
        }
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------ softmax, results
    // Threads of warps w and w + 4 share a row: half 0 takes tokens 0-63 of a
    // block and the first half of the dims, half 1 the others. A wait that
    // gave up does not end the loop, so that the halves keep meeting.
    const int half = warp >> 2, quad = warp & 3;
    const int wr = quad * 32 + lane;  // row of this block's half of the tile
    const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // TMEM lane field
    int nb = blocks0, seg = first;
    bool ok = ok0;
    // First pass over a q8 pool: a warp fetches the scales of K or V of 32 of a block's tokens, a lane a token's, and
    // looks at them a block later. (Elsewhere it costs 5-20 % of the time: the copying warp and the preparing ones
    // set the pace over a q8 pool.)
    // First pass over a q8 pool: a warp looks at the scales of K or V of 32 of a block's tokens, a lane at a token's, which
    // are on their way while it waits for the block's scores. (1-5 % of the time; 5-25 % with the copying or the
    // preparing warps, which set the pace over a q8 pool.)
    [[maybe_unused]] uint32_t scales[NS];
    [[maybe_unused]] auto fetch = [&](int b, int pages) {
      const int kv = quad & 1, k = quad >> 1, page = __shfl_sync(0xffffffffu, pages, 2 * k + lane / kPage);
#pragma unroll
      for (int w = 0; w < NS; ++w) scales[w] = 0;
      if (wk.has_page(page) && b * kBN + 64 * half + 32 * k + lane < wk.v.kv_len) {  // (below 2^31: check_pool)
        const int row = (page * a.pool.hkv + wk.h) * kPage + lane % kPage;
        token_scales<NS>(static_cast<const uint8_t*>(kv ? a.pool.v_scale : a.pool.k_scale) + static_cast<int64_t>(row) * (NS * 4), scales);
      }
    };
    [[maybe_unused]] auto look = [&] {
      if (any_large(scales)) atomicMin(&ms.large, wk.seg);
    };
    for (;; ++seg) {
      Segment& g = ms.segment[(seg + shift) & 1];
      if (warp == 0) {
        const bool more = take();
        if (lane == 0) g = Segment{wk.s, wk.h, wk.mt, wk.b0, wk.b1, more, wk.v, wk.t};
      }
      named_sync(5, 256);
      if (!g.more) break;
      wk.seg = seg;
      wk.s = g.s;
      wk.h = g.h;
      wk.mt = g.mt;
      wk.b0 = g.b0;
      wk.b1 = g.b1;
      wk.v = g.v;
      wk.t = g.t;
      const int r = rank * 128 + wr, r_warp = rank * 128 + quad * 32;
      const bool valid = r < wk.t.rows, warp_valid = r_warp < wk.t.rows;
      const int base_p = wk.v.kv_len - wk.v.q_len, last = wk.t.rows - 1;
      const RowOf at = row_of(wk.t, min(r, last), a.G, a.g_inv);
      const int p = base_p + at.tok;
      const int wp0 = base_p + row_of(wk.t, min(r_warp, last), a.G, a.g_inv).tok;
      const int wp1 = base_p + row_of(wk.t, min(r_warp + 31, last), a.G, a.g_inv).tok;
      float m = valid ? -INFINITY : 0.f, l = 0.f, c = 0.f;
      int pages = lane < 4 ? wk.entry(wk.t.block(wk.b0), 4 * half + lane) : 0;
      for (int i = wk.b0; i < wk.b1; ++i, ++nb) {
        const int b = wk.t.block(i);
        const uint32_t gone = __ballot_sync(0xffffffffu, !wk.has_page(pages)) & 0xfu;
        // the lane's tokens of the half (lane, lane + 32) that are large: bits 0, 1 for K, 2, 3 for V
        [[maybe_unused]] uint32_t large = 0;
        if constexpr (LARGE) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int page = __shfl_sync(0xffffffffu, pages, 2 * k + lane / kPage);
            if (!wk.has_page(page)) continue;
            const int64_t at = static_cast<int64_t>((page * a.pool.hkv + wk.h) * kPage + lane % kPage) * (NS * 4);
            large |= (large_token<NS>(static_cast<const uint8_t*>(a.pool.k_scale) + at) ? 1u : 0u) << k |
                     (large_token<NS>(static_cast<const uint8_t*>(a.pool.v_scale) + at) ? 4u : 0u) << k;
          }
        }
        [[maybe_unused]] auto large_bits = [&](int kv, int k) { return __ballot_sync(0xffffffffu, large >> (2 * kv + k) & 1); };
        if constexpr (Q8 && !LARGE) fetch(b, pages);
        if (i + 1 < wk.b1 && lane < 4) pages = wk.entry(wk.t.block(i + 1), 4 * half + lane);
        ok &= wait(ms.s_full[nb & 1], (nb >> 1) & 1);
        if constexpr (Q8 && !LARGE) look();
        tc_fence_after();
        if (warp_valid) {
          if (i == wk.b0 && valid)  // scale x log2(e) x 2^e, kept normal and finite so that -inf x c is -inf
            c = fminf(fmaxf(a.c * __uint_as_float(static_cast<uint32_t>(127 + ms.qe[(wk.seg + shift) % 3][wr]) << 23), 1.2e-38f), 3e38f);
          const uint32_t sa = tm + lanes + 256 + (nb & 1) * kBN;
          uint32_t x[32], y[32];
          uint32_t sx = 0xffffffffu, sy = 0xffffffffu;
          const bool part = gone || !block_full(b, wp0, wp1, a.window, a.sinks);
          if (part) {
            sx = seen_bits(p, b * kBN + 64 * half, a.window, a.sinks);
            sy = seen_bits(p, b * kBN + 64 * half + 32, a.window, a.sinks);
            if (gone & 1) sx &= 0xffff0000u;
            if (gone & 2) sx &= 0x0000ffffu;
            if (gone & 4) sy &= 0xffff0000u;
            if (gone & 8) sy &= 0x0000ffffu;
          }
          auto hide = [&](uint32_t (&v)[32], uint32_t seen) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(seen >> j & 1)) v[j] = 0xff800000u;  // -inf
          };
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto top = [&](const uint32_t (&v)[32]) {
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mx[j / 2 & 3] = fmaxf(fmaxf(mx[j / 2 & 3], __uint_as_float(v[j])), __uint_as_float(v[j + 1]));
          };
          tmem_ld32(sa + 64 * half, x);
          tmem_ld32(sa + 64 * half + 32, y);
          tmem_wait_ld(x);
          tmem_wait_ld(y);
          const float cb = LARGE ? 1.f : c;  // the scores times cb are the exponents
          if constexpr (LARGE) {
            auto exponents = [&](uint32_t (&v)[32], uint32_t k_large, uint32_t v_large) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                v[j] = __float_as_uint(fmaf(__uint_as_float(v[j]) * c, k_large >> j & 1 ? 256.f : 1.f, v_large >> j & 1 ? 8.f : 0.f));
            };
            exponents(x, large_bits(0, 0), large_bits(1, 0));
            exponents(y, large_bits(0, 1), large_bits(1, 1));
          }
          if (part) {
            hide(x, sx);
            hide(y, sy);
          }
          top(x);
          top(y);
          float my = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cb;  // cb > 0
          ms.swap[nb & 1][half][wr] = my;
          named_sync(1 + quad, 64);
          my = fmaxf(my, ms.swap[nb & 1][half ^ 1][wr]);
          if (__any_sync(0xffffffffu, my > m + kLazy)) {  // the same in both halves
            const float nm = fmaxf(m, my);
            const float f = nm == -INFINITY ? 1.f : ex2(m - nm);
            m = nm;
            l *= f;
            if (i > wk.b0) {  // rescale O, once the product before is done (these scores show that those before it are)
              ok &= wait(ms.pv_done, (nb - 1) & 1);
              tc_fence_after();
              uint32_t z[32];
#pragma unroll 1
              for (int k = half * NS; k < half * NS + NS; ++k) {
                tmem_ld32(tm + lanes + 32 * k, z);
                tmem_wait_ld(z);
#pragma unroll
                for (int j = 0; j < 32; ++j) z[j] = __float_as_uint(__uint_as_float(z[j]) * f);
                tmem_st32(tm + lanes + 32 * k, z);
              }
            }
          }
          const float mm = (m == -INFINITY ? 0.f : m) - kLift;
          const uint64_t c2 = pack2(cb, cb), m2 = pack2(-mm, -mm);
          uint64_t l2 = pack2(0.f, 0.f), l3 = l2;
          // P of the half lies over its own scores, which are in registers
          auto weigh = [&](const uint32_t (&v)[32], uint64_t& sum, uint32_t dst, [[maybe_unused]] uint32_t v_large) {
            uint32_t h[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), c2, m2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              h[j] = pack_half2(e0, e1);
              if constexpr (LARGE) {
                if (v_large >> (2 * j) & 1) e0 *= 0.00390625f;
                if (v_large >> (2 * j + 1) & 1) e1 *= 0.00390625f;
              }
              sum = add2(sum, pack2(e0, e1));
            }
            tmem_st16(dst, h);
          };
          weigh(x, l2, sa + 64 * half, LARGE ? large_bits(1, 0) : 0);
          weigh(y, l3, sa + 64 * half + 16, LARGE ? large_bits(1, 1) : 0);
          float a0, a1;
          unpack2(add2(l2, l3), a0, a1);
          l += a0 + a1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) lead_arrive(ms.p_ready[nb & 1]);
      }
      // the result of the segment: O, once its last product is done. (Not by
      // pv_done: a wait tells only two neighbouring phases apart, and here the
      // one before the last may be open as well as the last one over.)
      ok &= wait(ms.o_full, (wk.seg + shift) & 1);
      if constexpr (Q8 && !LARGE) named_sync(5, 256);  // what any warp noted is known to all
      if (!warp_valid) continue;
      tc_fence_after();
      ms.swap[nb & 1][half][wr] = l;  // (read there last two blocks ago)
      named_sync(1 + quad, 64);
      l += ms.swap[nb & 1][half ^ 1][wr];
      named_sync(1 + quad, 64);
      if (Q8 && !LARGE && *const_cast<volatile int*>(&ms.large) <= wk.seg) continue;  // left to the second pass
      const bool whole = wk.whole();
      const int slot = 2 * worker + (wk.seg == 0 ? 0 : 1);
      const int row = wk.v.r0 + at.tok, head = wk.h * a.G + at.head;
      const bool patch = *const_cast<volatile int*>(&ms.flag[(wk.seg + shift) & 3]) == wk.seg + shift + 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (!whole && valid && half == 0) a.ml[slot * M + r] = ok ? make_float2(m, l) : make_float2(0.f, NAN);
#pragma unroll 1
      for (int k = half * NS; k < half * NS + NS; ++k) {
        uint32_t x[32];
        float y[32];
        tmem_ld32(tm + lanes + 32 * k, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = ok ? __uint_as_float(x[j]) : NAN;
        if (valid && ok && patch) {
          // rows that see a cleared value add it: +-inf or NaN whatever its weight
          for (int i = wk.b0; i < wk.b1; ++i) {
            const int b = wk.t.block(i);
            for (int t = 0; t < kBN; ++t) {
              const int pg = wk.entry(b, t / kPage);
              if (!wk.has_page(pg) || !(seen_bits(p, b * kBN + (t & ~31), a.window, a.sinks) >> (t & 31) & 1)) continue;
              const int64_t e = ((static_cast<int64_t>(pg) * a.pool.hkv + wk.h) * kPage + t % kPage) * DH + 32 * k;
              if (Q8) {
                const float d = __half2float(static_cast<const __half*>(a.pool.v_scale)[e / 32]);
                if (isfinite(d)) continue;
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] += d * static_cast<float>(static_cast<const int8_t*>(a.pool.v)[e + j]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float d = __half2float(static_cast<const __half*>(a.pool.v)[e + j]);
                  if (!isfinite(d)) y[j] += d;
                }
              }
            }
          }
        }
        if (valid && !whole) {
          float* dst = a.part + (static_cast<int64_t>(slot) * M + r) * DH + 32 * k;
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + j), "f"(y[j]), "f"(y[j + 1]),
                         "f"(y[j + 2]), "f"(y[j + 3]), "f"(y[j + 4]), "f"(y[j + 5]), "f"(y[j + 6]), "f"(y[j + 7])
                         : "memory");
        } else if (valid) {
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = !ok ? NAN : l == 0.f ? 0.f : y[j] * inv;
          put_out<32>(a, row, head, 32 * k, y);
        }
        __syncwarp();
      }
      tc_fence_before();
    }
    if (Q8 && !LARGE && tid == 0) {
      ms.taken = seg;
      ms.blocks = nb;
    }
  } else {
    // ------------------------------------------------------ operand preparing
    const int pw = warp - kWarpPrep, pt = pw * 32 + lane;
    constexpr int kPT = kPrep * 32;
    int n = units0;
    bool ok = ok0;
    [[maybe_unused]] int turn = 0;  // warp whose turn it is to convert a box
    // unit u of K or V of block b: hand it over, converted (q8) and cleared (V
    // of a partly seen block). One body of code for K and V: more would not
    // stay in the instruction cache.
    auto unit = [&](int kv, int u, int b) {
      const int slot = n % C::kSlots, phase = (n / C::kSlots) & 1;
      [[maybe_unused]] const int rs = Q8 ? n % C::kRawSlots : 0, rphase = Q8 ? (n / C::kRawSlots) & 1 : 0;
      ++n;
      const int nkeys = kv ? C::kKeysV : C::kKeysK, nsl = kv ? C::kSlabsV : C::slabs_k(u);
      const int key0 = CG == 2 ? (kv ? 0 : 64 * rank) : (kv ? u * C::kKeysV : 0);
      uint8_t* const dst = ring + slot * C::kSlot;
      bool found = false;
      const bool partly = kv && !block_full(b, wk.t.p0, wk.t.p1, a.window, a.sinks);
      if constexpr (!Q8) {
        if (!wait(ms.full[slot], phase)) return false;
        if (partly) {
          const int end = wk.v.kv_len - b * kBN - key0;  // tokens from here on do not exist
#pragma unroll 4
          for (int q = pt; q < nkeys * nsl * 8; q += kPT) {
            uint4* ptr = reinterpret_cast<uint4*>(dst + q * 16);
            uint4 x = *ptr;
            const int key = q / (nsl * 128) * kPage + q / 8 % kPage;  // [page][slab][16][128 B]
            bool bad = false;
            uint32_t* w = &x.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((w[j] & 0x7c00u) == 0x7c00u) { w[j] &= 0xffff0000u; bad = true; }
              if ((w[j] & 0x7c000000u) == 0x7c000000u) { w[j] &= 0x0000ffffu; bad = true; }
            }
            if (key >= end) *ptr = make_uint4(0, 0, 0, 0);
            else if (bad) {
              *ptr = x;
              found = true;
            }
          }
          fence_async_shared();
        }
      } else {
        if (!wait(ms.raw_full[rs], rphase)) return false;
        if (!wait(ms.empty[slot], phase ^ 1)) return false;
        const int slab0 = CG == 2 ? (kv ? rank * C::kSlabsV : 0) : (kv ? 0 : 2 * u);
        const uint8_t* src = raw + rs * C::kRaw;
        const __half* sc = reinterpret_cast<const __half*>(src + C::kSlot / 2);
        const uint32_t gone = static_cast<uint32_t>(ms.raw_pages[rs]);
        const int end = partly ? wk.v.kv_len - b * kBN - key0 : nkeys;
        // A warp converts a box (16 tokens x kBox codes) at a time, 16 codes a
        // lane and step; the warps take the boxes of all units in turn.
        constexpr int kBC = C::kBox / 16, kTok = 32 / kBC, kSteps = kPage / kTok;
        const int nbx = nsl * 64 / C::kBox, boxes = nkeys / kPage * nbx, inv = 256 / nbx + 1;
        const int cc = lane % kBC, tok0 = lane / kBC;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        int pb = pw - turn;
        if (pb < 0) pb += kPrep;
        turn = (turn + boxes) % kPrep;
#pragma unroll 1
        for (; pb < boxes; pb += kPrep) {
          const int page = (pb * inv) >> 8, dim = (pb - page * nbx) * C::kBox + cc * 16;
          const int sl = dim / 64, ch = (dim % 64) / 8;
          uint4 codes[kSteps];
          __half d[kSteps];
#pragma unroll
          for (int t = 0; t < kSteps; ++t) {
            codes[t] = *reinterpret_cast<const uint4*>(src + pb * (kPage * C::kBox) + t * 512 + lane * 16);
            d[t] = sc[(page * kPage + tok0 + t * kTok) * (2 * NS) + (slab0 * 64 + dim) / 32];
          }
          // K: [8 tokens][slab][8][128 B], V: [page][slab][16][128 B]
          const int group = kv ? 1024 : C::kBoxSlabsK * 1024;  // from tokens 0-7 of the page to 8-15
          uint8_t* const slab = dst + page * kPage * 128 * (kv ? C::kSlabsV : C::kBoxSlabsK) + sl * (kv ? 2048 : 1024);
#pragma unroll
          for (int t = 0; t < kSteps; ++t) {
            const int tok = tok0 + t * kTok;
            uint32_t o[8];
            const uint32_t cw[4] = {codes[t].x, codes[t].y, codes[t].z, codes[t].w};
            const __half2 d2 = __half2half2(d[t]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w = cw[j] ^ 0x80808080u;  // code + 128; 0x6400 | byte is 1024 + byte
              const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
              const __half2 a2 = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&lo), off), d2);
              const __half2 b2 = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&hi), off), d2);
              o[2 * j] = *reinterpret_cast<const uint32_t*>(&a2);
              o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            // (the rows of neighbouring slabs share banks: exchanging the two pieces of every other lane avoids that
            // and costs more than it saves, 74 against 70 us for 4 x 3 rows over 23K tokens)
            uint8_t* row = slab + (tok >> 3) * group + (tok & 7) * 128;
            *reinterpret_cast<uint4*>(row + ((ch ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (tok & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          if constexpr (LARGE) {  // 2^-8 of the values of large tokens, in place of what was stored
            const uint32_t large = __ballot_sync(0xffffffffu, large_token<NS>(src + C::kSlot / 2 + (page * kPage + lane % kPage) * (NS * 4)));
            const __half2 small = __half2half2(__ushort_as_half(0x1c00));
#pragma unroll 1
            for (int t = 0; t < kSteps; ++t) {
              const int tok = tok0 + t * kTok;
              if (!(large >> tok & 1)) continue;
              const uint4 code = *reinterpret_cast<const uint4*>(src + pb * (kPage * C::kBox) + t * 512 + lane * 16);
              const __half2 d2 = __half2half2(sc[(page * kPage + tok) * (2 * NS) + (slab0 * 64 + dim) / 32]);
              const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
              uint32_t o[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t w = cw[j] ^ 0x80808080u;
                const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
                const __half2 a2 = __hmul2(__hmul2(__hsub2(*reinterpret_cast<const __half2*>(&lo), off), small), d2);
                const __half2 b2 = __hmul2(__hmul2(__hsub2(*reinterpret_cast<const __half2*>(&hi), off), small), d2);
                o[2 * j] = *reinterpret_cast<const uint32_t*>(&a2);
                o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              uint8_t* row = slab + (tok >> 3) * group + (tok & 7) * 128;
              *reinterpret_cast<uint4*>(row + ((ch ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (tok & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
          if (gone || partly) {  // missing pages read as zeros, unseen V values too
#pragma unroll 1
            for (int t = 0; t < kSteps; ++t) {
              const int tok = tok0 + t * kTok, key = page * kPage + tok;
              const uint32_t scale = __half_as_ushort(sc[key * (2 * NS) + (slab0 * 64 + dim) / 32]);
              const bool none = gone >> page & 1;
              const bool bad = partly && !none && key < end && (scale & 0x7c00u) == 0x7c00u;
              if (none || bad || (kv && key >= end)) {
                uint8_t* row = slab + (tok >> 3) * group + (tok & 7) * 128;
                *reinterpret_cast<uint4*>(row + ((ch ^ (tok & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (tok & 7)) << 4)) = make_uint4(0, 0, 0, 0);
              }
              found |= bad;
            }
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(ms.raw_empty[rs]));
      }
      if (found) {
        if (CG == 1) {
          *const_cast<volatile int*>(&ms.flag[(wk.seg + shift) & 3]) = wk.seg + shift + 1;
        } else {
          for (int k = 0; k < 2; ++k) st_cluster(peer_addr(smem_u32(&ms.flag[(wk.seg + shift) & 3]), k), wk.seg + shift + 1);
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
        }
      }
      __syncwarp();
      if (lane == 0) lead_arrive(ms.ready[slot]);
      return true;
    };
    constexpr int kLPR = NS == 3 ? 32 : 8 * NS;  // lanes per row of Q
    constexpr int kRPP = 32 / kLPR;              // rows per warp and pass
    constexpr int kPass = (128 + kPrep * kRPP - 1) / (kPrep * kRPP), kBatch = kPass < 11 ? kPass : 11;
    const int ch = lane % kLPR, sub = lane / kLPR;
    while (ok && take()) {
      // Q of the tile: the first rows are fetched before the products of the
      // segment before are known to no longer read it, and stored after that
      const int rows = min(128, wk.t.rows - rank * 128);
#pragma unroll 1
      for (int pass = 0; pass < kPass; pass += kBatch) {
        // Addresses are clamped to valid rows and columns rather than the loads
        // made conditional: all of a batch are in flight at once.
        uint32_t o[kBatch][4];
        auto row_ptr = [&](int t) {
          const int r = min(((pass + t) * kPrep + pw) * kRPP + sub, max(rows, 1) - 1);
          const RowOf at = row_of(wk.t, min(rank * 128 + r, wk.t.rows - 1), a.G, a.g_inv);
          return static_cast<const uint16_t*>(a.q.data) + (wk.v.r0 + at.tok) * a.q.row_stride +
                 (wk.h * a.G + at.head) * a.q.head_stride + min(ch, 8 * NS - 1) * 8;
        };
        if (a.vq) {
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            if (t >= 2 && (pass + t) * kPrep * kRPP >= rows) break;
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(row_ptr(t)));
            o[t][0] = x.x; o[t][1] = x.y; o[t][2] = x.z; o[t][3] = x.w;
          }
        } else {
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            const uint16_t* qp = row_ptr(t);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][j] = qp[2 * j] | static_cast<uint32_t>(qp[2 * j + 1]) << 16;
          }
        }
        if (pass == 0 && wk.seg + shift > 0) ok = wait(ms.q_free, (wk.seg + shift - 1) & 1);
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
          const int r0 = ((pass + t) * kPrep + pw) * kRPP, r = r0 + sub;
          if (r0 >= rows) break;  // whole warps
          int e = 0;
          if (a.dtype == MK_BF16) {
            // the row times a power of two that brings its largest value to [2^14, 2^15): exact for what is at least
            // 2^-31 of it, to 2^-25 for the rest (2^-39 of the largest); infinite and NaN values stay
            // (magnitudes compared as integers; a row's lanes in one reduction)
            float x[8];
            uint32_t top2 = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[2 * j] = __uint_as_float(o[t][j] << 16);
              x[2 * j + 1] = __uint_as_float(o[t][j] & 0xffff0000u);
              top2 = __vmaxu2(top2, o[t][j] & 0x7fff7fffu);
            }
            const uint32_t group = kLPR == 32 ? 0xffffffffu : ((1u << kLPR % 32) - 1) << (sub * kLPR);
            const uint32_t mx = __reduce_max_sync(group, max(top2 & 0xffffu, top2 >> 16));
            e = max(static_cast<int>(mx >> 7) - (127 + 14), -126);  // at most 114; 2^e and 2^-e are normal
            const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][j] = pack_half2(x[2 * j] * f, x[2 * j + 1] * f);
          }
          if (r < rows && ch < 8 * NS)
            *reinterpret_cast<uint4*>(sq + (ch / 8) * 16384 + r * 128 + (((ch % 8) ^ (r & 7)) << 4)) =
                make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
          if (ch == 0 && r < rows) ms.qe[(wk.seg + shift) % 3][r] = static_cast<int8_t>(e);
        }
      }
      if (!ok) break;
      fence_async_shared();
      __syncwarp();
      if (lane == 0) lead_arrive(ms.q_ready);
      if (a.gate.data) {  // the gate's rows on their way to L2
        for (int k = pt; k < rows * NS; k += kPT) {
          const RowOf at = row_of(wk.t, rank * 128 + k / NS, a.G, a.g_inv);
          const uint16_t* line = static_cast<const uint16_t*>(a.gate.data) + (wk.v.r0 + at.tok) * a.gate.row_stride +
                                 (wk.h * a.G + at.head) * a.gate.head_stride + k % NS * 64;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
        }
      }
      if (wk.more()) {  // the next tile's rows on their way to L2
        const bool wrap = wk.mt + 1 == wk.n_mt;
        const int h = wk.h + wrap, R0 = (wrap ? 0 : wk.mt + 1) * M + rank * 128;
        const int left_rows = h < a.pool.hkv ? min(128, wk.v.q_len * a.G - R0) : 0;
        const int t0 = R0 / a.G, h0 = R0 - t0 * a.G;
        for (int k = pt; k < left_rows * NS; k += kPT) {
          const int x = h0 + k / NS, q = (x * a.g_inv) >> 20;
          const uint16_t* line = static_cast<const uint16_t*>(a.q.data) + (wk.v.r0 + t0 + q) * a.q.row_stride +
                                 (h * a.G + x - q * a.G) * a.q.head_stride + k % NS * 64;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
        }
      }
      for (int i = wk.b0; ok && i <= wk.b1; ++i) {
        if (i < wk.b1)
          for (int u = 0; ok && u < C::KU; ++u) ok = unit(0, u, wk.t.block(i));
        if (i > wk.b0)
          for (int u = 0; ok && u < C::VU; ++u) ok = unit(1, u, wk.t.block(i - 1));
      }
    }
    if (Q8 && !LARGE && pt == 0) ms.units = n;
  }
}

// (A function of its own: inlined it took registers from the first pass, 3 % of the time over q8 pools.)
template <int NS, int CG>
__device__ __noinline__ void large_pass(const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv, uint8_t* smem, uint32_t tm) {
  attend_pass<NS, true, CG, true>(a, tk, tv, smem, tm);
}

template <int NS, bool Q8, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams a, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv) {
  using C = Cfg<NS, Q8, CG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const ring = smem + C::kQ;
  Misc& ms = *reinterpret_cast<Misc*>(ring + C::kSlots * C::kSlot + C::kRawSlots * C::kRaw);
  const int tid = threadIdx.x, warp = tid / 32;
  const int rank = CG == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  // all warps (of both blocks): what they did to shared and tensor memory is done
  auto meet = [] {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      bar_init(bar(ms.full[i]), 1);
      bar_init(bar(ms.ready[i]), CG * kPrep);
      bar_init(bar(ms.empty[i]), 1);
    }
    for (int i = 0; i < C::kRawSlots; ++i) {
      bar_init(bar(ms.raw_full[i]), 1);
      bar_init(bar(ms.raw_empty[i]), kPrep);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(ms.s_full[i]), 1);
      bar_init(bar(ms.p_ready[i]), 8 * CG);
    }
    bar_init(bar(ms.pv_done), 1);
    bar_init(bar(ms.o_full), 1);
    bar_init(bar(ms.q_ready), CG * kPrep + (static_cast<int>(blockIdx.x / CG) == a.skip));  // (an arrival that never comes)
    bar_init(bar(ms.q_free), 1);
    bar_init(bar(ms.drained), 1);
    ms.dead[0] = (smem_u32(smem) & 1023u) != 0;  // (the swizzled tiles need the alignment)
    ms.dead[1] = a.wait_us;
    ms.failed = 0;
    for (int i = 0; i < 4; ++i) ms.flag[i] = 0;
    ms.large = INT_MAX;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) tmem_alloc<CG>(smem_u32(&ms.tmem), 512);
  find_start<C::M>(a, reinterpret_cast<int*>(ring), &ms.start, blockIdx.x / CG, rank == 0);
  fence_async_shared();  // the scratch lay where tensor copies go
  meet();
  tc_fence_after();
  const uint32_t tm = ms.tmem;
  asm volatile("griddepcontrol.launch_dependents;");
  attend_pass<NS, Q8, CG, false>(a, tk, tv, smem, tm);
  if constexpr (Q8 && CG == 2) {  // both blocks of a pair go on alike, even if the pool changes under the kernel
    __syncthreads();
    if (threadIdx.x == 0) min_cluster(peer_addr(smem_u32(&ms.large), static_cast<uint32_t>(~blockIdx.x & 1)), ms.large);
  }
  meet();
  if constexpr (Q8) {
    if (ms.large != INT_MAX) {
      tc_fence_after();
      large_pass<NS, CG>(a, tk, tv, smem, tm);
      meet();
    }
  }
  if (*const_cast<volatile int*>(&ms.failed)) {
    if (warp == kWarpMma) bar_drain(bar(ms.drained), 0);
    meet();
  }
  if (warp == kWarpMma) tmem_free<CG>(tm, 512);
}

// ------------------------------------------------------------------- launch
// Blocks (pairs) that are resident at once, found once per device; 0 on error.
template <int NS, bool Q8, int CG>
int resident_workers(int device) {
  using C = Cfg<NS, Q8, CG>;
  static std::atomic<int> known[64];
  if (device < 0 || device >= 64) return 0;
  int n = known[device].load();
  if (n) return n;
  const auto fn = attend_kernel<NS, Q8, CG>;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return 0;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
  n = sms;
  if (CG == 2) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {2, 1, 1};
    cfg.gridDim = dim3(2 * (sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) return 0;
  }
  if (n > kMaxWorkers / CG) n = kMaxWorkers / CG;
  known[device].store(n);
  return n;
}

template <int NS, bool Q8, int CG>
cudaError_t launch_attend(AttendParams a, const CUtensorMap& tk, const CUtensorMap& tv, int device, cudaStream_t stream) {
  using C = Cfg<NS, Q8, CG>;
  a.workers = resident_workers<NS, Q8, CG>(device);
  if (!a.workers) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {CG, 1, 1};
  cfg.gridDim = dim3(a.workers * CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel<NS, Q8, CG>, a, tk, tv);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t jc{};
  cudaLaunchAttribute ja[1];
  ja[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  ja[0].val.programmaticStreamSerializationAllowed = 1;
  jc.gridDim = dim3(a.workers, kJoinSplit);
  jc.blockDim = dim3(256);
  jc.stream = stream;
  jc.attrs = ja;
  jc.numAttrs = 1;
  return cudaLaunchKernelEx(&jc, attend_join<NS, CG>, a);
}

template <bool Q8>
cudaError_t launch_any(int ns, int cg, const AttendParams& a, const CUtensorMap& tk, const CUtensorMap& tv, int device,
                       cudaStream_t stream) {
  switch (ns * 2 + (cg - 1)) {
    case 2: return launch_attend<1, Q8, 1>(a, tk, tv, device, stream);
    case 4: return launch_attend<2, Q8, 1>(a, tk, tv, device, stream);
    case 5: return launch_attend<2, Q8, 2>(a, tk, tv, device, stream);
    case 6: return launch_attend<3, Q8, 1>(a, tk, tv, device, stream);
    case 8: return launch_attend<4, Q8, 1>(a, tk, tv, device, stream);
    case 9: return launch_attend<4, Q8, 2>(a, tk, tv, device, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ops
}  // namespace mk
