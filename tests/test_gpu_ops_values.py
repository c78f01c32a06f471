"""Attention over values at the ends of the types' ranges, against the 64-bit reference of
tests/ops_helpers.py: weights far below a row's largest; bf16
queries of every magnitude the type has."""
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
