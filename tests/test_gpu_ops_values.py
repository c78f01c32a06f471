"""Attention over values at the ends of the types' ranges, against the 64-bit reference of
tests/ops_helpers.py: q8 blocks past binary16's largest value, seen and unseen; weights far below
a row's largest; bf16 queries of every magnitude the type has."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import Case, assert_within  # noqa: E402


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def attend(ops, c, **kw):
    pool, rows = c.ops()
    return ops.attend(pool, rows, c.q, **kw)[:c.rows_used]


# ------------------------------------------------- q8 values past binary16
def _put(c, name, seq, pos, head, block, scale, codes):
    """One q8 block of a cached token: 32 codes and their scale (binary16)."""
    page, slot, dims = int(c.tables[seq, pos // 16]), pos % 16, slice(32 * block, 32 * block + 32)
    codes = codes.to(torch.int8).cuda()
    d = torch.tensor(scale).half().cuda()
    c.pool[name][page, head, slot, dims] = codes
    c.pool[name + "_scale"][page, head, slot, block] = d
    c.value[name][page, head, slot, dims] = codes.double() * d.double()


LARGE = [([(150, 400), (3, 700), (1, 33)], 6, 2, 64), ([(2, 90), (140, 300)], 4, 2, 128), ([(70, 150), (4, 500)], 3, 1, 192),
         ([(60, 333), (1, 40)], 12, 2, 256), ([(3, 1000), (1, 129)], 12, 2, 256)]


@pytest.mark.parametrize("amp", [1e5, 1.5e6])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("seqs,hq,hkv,dh", LARGE)
def test_q8_pools_of_large_values(ops, seqs, hq, hkv, dh, window, sinks, amp):
    """Every block's scale is past 516, where 127 codes leave binary16."""
    c = Case(seqs, hq, hkv, dh, "q8", "bf16", seed=40, amp=amp)
    s = 1.0 / (amp * math.sqrt(dh))  # scores of ordinary size
    got = attend(ops, c, window=window, sinks=sinks, scale=s)
    assert_within(got, *c.attend_ref(window, sinks, scale=s))


@pytest.mark.parametrize("scale,dtype", [(511.5, "f16"), (516.0, "f16"), (600.0, "f16"), (511.5, "bf16"), (516.0, "bf16"), (8000.0, "bf16"),
                                         (65504.0, "bf16")])
@pytest.mark.parametrize("dh,hq,hkv,n", [(64, 4, 2, 40), (128, 4, 1, 90), (192, 2, 1, 150), (256, 6, 1, 60), (256, 6, 1, 3)])
def test_q8_large_blocks_seen_and_unseen(ops, dh, hq, hkv, n, scale, dtype):
    """Some blocks of a few tokens are large. Rows that see them give the definition's values; the
    others are as if the tokens were not there (their bound knows nothing of the large values)."""
    first, window = 60, 25
    c = Case([(n, n + first), (2, 50)], hq, hkv, dh, "q8", dtype, seed=41, pad_rows=0)
    g = torch.Generator().manual_seed(42)
    codes = torch.randint(-127, 128, (32,), generator=g)
    codes[0], codes[1], codes[2] = 127, -127, -128
    block = dh // 32 - 1
    # the queries are small where K is large, so that the scores stay of ordinary size
    c.q[..., 32 * block:] = (c.q[..., 32 * block:].float() * (2.0 / (scale * 127))).to(c.dtype)
    large = [first + n - 2, first + n // 2, 5]  # seen by the last rows, by the later half, outside most windows
    for pos in large:
        _put(c, "v", 0, pos, 0, 0, scale, codes)
        _put(c, "k", 0, pos, hkv - 1, block, scale, codes)
    for window in (0, window):
        got = attend(ops, c, window=window)
        want, bound = c.attend_ref(window)
        assert_within(got, want, bound)
        was = c.value["v"]
        c.value["v"] = was.clone()
        for pos in large:
            c.value["v"][int(c.tables[0, pos // 16]), 0, pos % 16, :32] = 0
        want, bound = c.attend_ref(window)
        c.value["v"] = was
        p = torch.arange(first, first + n)
        sees = torch.zeros(n, dtype=torch.bool)
        for pos in large:
            sees |= (pos <= p) & ((p - pos < window) if window else True)
        blind = torch.cat([~sees, torch.ones(2, dtype=torch.bool)]).cuda()  # the second sequence too
        assert window == 0 or n < 30 or int(blind.sum()) > 5
        assert_within(got[blind], want[blind], bound[blind])


@pytest.mark.parametrize("n", [1, 5, 100])
def test_q8_large_tokens_all_over_a_long_context(ops, n):
    """Every tenth token has large blocks of V, every seventh of K, of all sizes up to the largest scale."""
    T, dh = 3000, 256
    c = Case([(n, T)], 6, 1, dh, "q8", "bf16", seed=43)
    page, slot = c.tables[0].long().repeat_interleave(16)[:T], torch.arange(T, device="cuda") % 16
    g = torch.Generator().manual_seed(44)
    for name, step, block in (("v", 10, 3), ("k", 7, 0)):
        t = torch.arange(0, T, step)
        d = (512 * 127 ** torch.rand(len(t), generator=g)).half().cuda()
        P, S = page[t], slot[t]
        c.pool[name + "_scale"][P, 0, S, block] = d
        dims = slice(32 * block, 32 * block + 32)
        c.value[name][P, 0, S, dims] = c.pool[name][P, 0, S, dims].double() * d.double()[:, None]
    c.q[..., :32] = (c.q[..., :32].float() * 1e-6).to(c.dtype)
    assert_within(attend(ops, c), *c.attend_ref())
    assert_within(attend(ops, c, window=700, sinks=30), *c.attend_ref(700, 30))


@pytest.mark.parametrize("n,count,dh,hq,hkv", [(1, 400, 64, 4, 2), (3, 250, 256, 6, 1), (100, 24, 128, 4, 2)])
def test_q8_large_tokens_in_some_of_many_sequences(ops, n, count, dh, hq, hkv):
    """Blocks take several sequences each, and cut them: results before the first large value, behind it
    and across the cuts, into an output of their own, over the queries and over the gate."""
    c = Case([(min(n, 20 + 37 * i % 400), 20 + 37 * i % 400) for i in range(count)], hq, hkv, dh, "q8", "bf16", seed=50, pad_rows=3)
    g = torch.Generator().manual_seed(51)
    codes = torch.randint(-127, 128, (32,), generator=g)
    for i in (count // 3, count // 3 + 1, count - 1):
        T = c.seqs[i][1]
        for pos in (0, T // 2, T - 1):
            _put(c, "v", i, pos, hkv - 1, 1, 3000.0 + i, codes)
            _put(c, "k", i, pos, 0, 0, 900.0, codes)
    c.q[..., :32] = (c.q[..., :32].float() * 2e-5).to(c.dtype)
    pool, rows = c.ops()
    q, gate = c.q.clone(), c.gate.clone()
    for out in (torch.full_like(q, 5.0), c.q, c.gate):
        behind = out[c.rows_used:].clone()
        got = ops.attend(pool, rows, c.q, gate=c.gate, out=out)
        assert torch.equal(got[c.rows_used:], behind)
        got = got[:c.rows_used].clone()
        c.q.copy_(q)
        c.gate.copy_(gate)
        assert_within(got, *c.attend_ref(gate=True))


@pytest.mark.parametrize("n", [1, 40])
def test_q8_scales_that_are_no_numbers_in_unused_places(ops, n):
    """What lies behind a sequence's end or on no page of it changes nothing, not even a bit."""
    c = Case([(n, 333), (1, 17)], 6, 1, 256, "q8", "f16", seed=52)
    want = attend(ops, c)
    for name in ("k_scale", "v_scale"):
        s = c.pool[name]
        s[torch.isnan(s)] = 60000.0
    assert torch.equal(attend(ops, c), want)


# ------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 18.0, 20.0, 22.0])
@pytest.mark.parametrize("n,hq,dh,at,copies", [(1, 6, 256, 0, 200), (3, 6, 256, 70, 160), (150, 2, 128, 0, 100), (2, 4, 64, 11990, 200),
                                                (100, 3, 256, 5, 90)])
def test_a_dominant_token_without_a_value(ops, n, hq, dh, at, copies, gap, dtype, kv):
    """As many sequences over the same pages as leave each of them in one piece. One token takes nearly all the weight and its V is zero: the output is the sum of 12,000 small
    weights. Their error, with w the exact weight (at most 1) and P its binary16 value, which is kept
    2^11 above the row's largest weight: P is rounded by 2^-11 w, and by half of binary16's
    smallest step where it is subnormal, 2^-25 / 2^11 = 2^-36. V of a q8 pool is rounded by 2^-11,
    four fp32 roundings of scores up to 22 log2(e) give 4 2^-24 32 ln 2 < 2^-17."""
    T = 12000
    c = Case([(n, T)], hq, 1, dh, kv, dtype, seed=45, pad_rows=0)
    many = ops.KVRows(torch.arange(0, (copies + 1) * n, n, dtype=torch.int32, device="cuda"), c.kv_len.repeat(copies),
                      c.tables.repeat(copies, 1), copies * n, n)
    page, slot = c.tables[0].long().repeat_interleave(16)[:T], torch.arange(T, device="cuda") % 16
    for name, x in (("k", torch.zeros(T, dh)), ("v", 1 + 0.25 * torch.randn(T, dh, generator=torch.Generator().manual_seed(46)))):
        x = x.cuda()
        if name == "k":
            x[at, 0] = 8.0
        else:
            x[at] = 0
        if kv == "f16":
            c.pool[name][page, 0, slot] = x.half()
            c.value[name][page, 0, slot] = x.half().double()
        else:
            d = (x.unflatten(-1, (-1, 32)).abs().amax(-1) / 127).half()
            q = torch.where(d[..., None] > 0, (x.unflatten(-1, (-1, 32)) / d.float()[..., None]).round(), 0.0).clamp(-127, 127)
            c.pool[name][page, 0, slot] = q.flatten(-2).to(torch.int8)
            c.pool[name + "_scale"][page, 0, slot] = d
            c.value[name][page, 0, slot] = (q.double() * d.double()[..., None]).flatten(-2)
    c.q.zero_()
    c.q[..., 0] = 1.0
    s = gap / float(c.value["k"][page[at], 0, slot[at], 0])
    got = ops.attend(c.ops()[0], many, c.q.repeat(copies, 1, 1), scale=s).view(copies, n, hq, dh)
    v = c.gather(0, "v")[0][:, 0]
    for i in range(n):
        seen = T - n + i + 1
        w = torch.full((seen,), math.exp(-gap), dtype=torch.double, device="cuda")
        if at < seen:
            w[at] = 1.0
        w /= w.sum()
        want = w @ v[:seen]
        u = 2.0 ** -11
        rel = u + (u if kv == "q8" else 0.0) + 2.0 ** -17
        # each addition into the fp32 sums is cut at 2^-23 of the partial sum
        err = (rel + T * 2.0 ** -23) * (w @ v[:seen].abs()) + 2.0 ** -36 * v[:seen].abs().sum(0)
        step = torch.finfo(c.dtype).eps / 2
        bound = err + (want.abs() + err) * step + (2.0 ** -25 if dtype == "f16" else 0.0)
        assert_within(got[:, i], want.expand(copies, hq, dh), bound.expand(copies, hq, dh))


# ------------------------------------------------------------- bf16 queries
@pytest.mark.parametrize("e", [-126, -120, -105, 90, 116, 122])
@pytest.mark.parametrize("n,dh,hq,hkv", [(9, 128, 4, 2), (1, 64, 2, 1), (60, 256, 6, 1)])
def test_bf16_queries_to_the_ends_of_the_type(ops, n, dh, hq, hkv, e):
    """Queries about 2^e; the score scale undoes it, so the scores are of ordinary size."""
    c = Case([(n, 200)], hq, hkv, dh, "f16", "bf16", seed=47)
    c.q.copy_((c.q.double() * 2.0 ** e).to(torch.bfloat16))
    assert bool(torch.isfinite(c.q).all())
    s = 2.0 ** -e / math.sqrt(dh)
    assert_within(attend(ops, c, scale=s), *c.attend_ref(scale=s))


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -16, 2.0 ** -18, 2.0 ** -20, 2.0 ** -22])
@pytest.mark.parametrize("n,dh,hq", [(1, 128, 2), (80, 256, 6), (5, 64, 4)])
def test_bf16_queries_of_wide_spread(ops, n, dh, hq, small, kv):
    """One dim of a query is far larger than the others, where K is large: all of them count in the scores."""
    c = Case([(n, 300)], hq, 1, dh, kv, "bf16", seed=48)
    big = 4.0 * 2.0 ** -12 / small
    c.q[..., 1:] = (c.q[..., 1:].float() * small).to(torch.bfloat16)
    if kv == "f16":
        c.pool["k"][..., 1:] *= big
        c.pool["k"][..., 0] *= 2.0 ** -10
        c.value["k"] = c.pool["k"].double()
    else:  # a power of two on every scale but the first block's
        c.pool["k_scale"][..., 1:] *= big
        c.pool["k"][..., 0] = 1
        c.value["k"] = (c.pool["k"].double().unflatten(-1, (-1, 32)) * c.pool["k_scale"].double()[..., None]).flatten(-2)
    s = 2.0 ** 9 / math.sqrt(dh)
    assert_within(attend(ops, c, scale=s), *c.attend_ref(scale=s))


def test_bf16_queries_with_infinities(ops):
    """An infinite query makes the scores infinite by the signs of K: of tokens with -inf scores alone the
    row gives 0; any +inf gives NaN."""
    c = Case([(4, 40)], 2, 1, 64, "f16", "bf16", seed=49)
    c.pool["k"][..., 0] = -c.pool["k"][..., 0].abs() - 1
    c.value["k"] = c.pool["k"].double()
    c.q[1, 0, 0] = math.inf
    c.q[1, 0, 1:] = 2.0 ** 100  # far past binary16: the row's infinity must stay its only one
    c.q[2, 1, 0] = -math.inf
    c.q[3, 0, 5] = math.nan
    got = attend(ops, c)
    assert not got[1, 0].any()
    assert bool(torch.isnan(got[2, 1]).all()) and bool(torch.isnan(got[3, 0]).all())
    want, bound = c.attend_ref()
    for i, h in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 1)):
        assert_within(got[i, h], want[i, h], bound[i, h])
