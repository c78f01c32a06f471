"""Operators on trees of drafts on the GPU against 64-bit references
(tests/tree_helpers.py): norm, rotation and write; attention of nodes over the
cache and their ancestors; greedy acceptance; kept and copied tokens; all of
them together, in captured graphs, on other streams and on an engine's pool."""
import math
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import assert_within, half_even, q8_values  # noqa: E402
from tree_helpers import TreeCase, random_parents, turned, walk  # noqa: E402

EPS = 1e-6


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def bits(t):
    return t.view(torch.int16) if t.dtype in (torch.float16, torch.bfloat16) else t


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --------------------------------------------------- norm, rotation and write
def freqs(dims, base=1e7):
    return base ** (-torch.arange(dims // 2, dtype=torch.double, device="cuda") * 2 / max(dims, 1))


def rounded(bound, want, dtype):
    """The bound of a value that is then rounded once to dtype."""
    f = torch.finfo(dtype)
    return bound + (want.abs() + bound) * (f.eps / 2) + f.smallest_normal * f.eps


def check_rope(ops, c, rot, gains=(True, True), q=None, k=None, v=None, out=None, parents=None, positions=None, base=1e7):
    gain = [(0.5 + torch.rand(c.dh, device="cuda")) if g else None for g in gains]
    rope = ops.Rope(rot, base, *gain, eps=EPS, device="cuda")
    pool, rows = c.ops()
    before = {n: t.clone() for n, t in c.pool.items()}
    q = c.q if q is None else q
    k, v = c.new_k if k is None else k, c.new_v if v is None else v
    q0, k0 = q.clone(), k.clone()
    got = ops.rope_write(pool, rows, rope, q, k, v, parents=parents, positions=positions, out=out)
    assert out is None or got is out
    pos, used = [], torch.zeros(c.n_pages, 16, dtype=torch.bool, device="cuda")
    for i, (n, T) in enumerate(c.seqs):
        pos += c.positions(i) if parents is not None else list(range(T - n, T))
    if positions is not None:
        pos = positions[:c.rows_used].tolist()
    fr = freqs(rot, base)
    u = c.rows_used
    want, b = turned(q0[:u], pos, rot, fr, gain[0], EPS)
    assert_within(got[:u], want, rounded(b, want, c.dtype))
    if out is not None:  # rows of no sequence
        assert torch.equal(bits(got[u:]), bits(q0[u:]))
    wk, bk = turned(k0[:u], pos, rot, fr, gain[1], EPS)
    for i, (n, T) in enumerate(c.seqs):
        for j in range(n):
            slot = T - n + j
            page = int(c.tables[i, slot // 16]) if slot >= 0 else -1
            if not 0 <= page < c.n_pages:
                continue
            used[page, slot % 16] = True
            r = int(c.start[i]) + j
            for name, x, bd in (("k", wk[r], bk[r]), ("v", v[r].double(), torch.zeros_like(bk[r]))):
                row = c.pool[name][page, :, slot % 16].double()
                if c.kv == "f16":
                    assert_within(row, x, rounded(bd, x, torch.float16))
                    continue
                # a code is the nearest to x / d; d is half_even(amax / 127) up to the bound on amax
                d = c.pool[name + "_scale"][page, :, slot % 16].double()
                ax, ab = x.unflatten(-1, (-1, 32)).abs().amax(-1) / 127, bd.unflatten(-1, (-1, 32)).amax(-1) / 127
                assert bool((d >= half_even((ax - ab).clamp_min(0))).all()) and bool((d <= half_even(ax + ab)).all())
                d32 = d.repeat_interleave(32, -1)
                err = (row * d32 - x).abs()
                # nearest code, clamped at 127: the scale was rounded by up to half a binary16 step (or half its least one)
                assert bool((err <= d32 / 2 * (1 + 1e-12) + 127 * (d32 * 2.0 ** -11 + 2.0 ** -25) + bd).all())
                inner = row.abs() < 127
                assert bool((err <= d32 / 2 * (1 + 1e-12) + bd)[inner].all())
    for name, was in before.items():
        assert torch.equal(bits(c.pool[name].transpose(1, 2))[~used], bits(was.transpose(1, 2))[~used]), name
    return got


ROPES = [([(1, 1)], 1, 1, 64, 64), ([(1, 17), (3, 3), (16, 32)], 6, 2, 128, 64), ([(7, 40), (0, 5), (33, 33)], 3, 3, 192, 192),
         ([(130, 1000), (1, 16)], 24, 4, 256, 256), ([(5, 9)], 5, 1, 192, 128), ([(9, 30)], 4, 4, 256, 0)]


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("seqs,hq,hkv,dh,rot", ROPES)
def test_rope_write(ops, seqs, hq, hkv, dh, rot, dtype, kv):
    c = TreeCase(seqs, hq, hkv, dh, kv, dtype, seed=1)
    check_rope(ops, c, rot, parents=c.parents if rot != 128 else None)


@pytest.mark.parametrize("gains", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("kind", ["forest", "chain", "star"])
def test_rope_write_gains_and_trees(ops, gains, kind):
    c = TreeCase([(20, 300), (1, 1), (40, 40)], 6, 2, 128, "f16", "bf16", seed=2, kind=kind)
    check_rope(ops, c, 128, gains, parents=c.parents)


def test_rope_write_far_and_negative_positions(ops):
    """Angles of positions up to 32 bits: a 32-bit product would be off by hundreds of radians."""
    c = TreeCase([(40, 64)], 2, 1, 64, "f16", "f32", seed=3)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 123456789, 96000, -77] + list(range(10 ** 9, 10 ** 9 + 33))
    check_rope(ops, c, 64, (False, False), positions=i32(pos))
    check_rope(ops, c, 64, (False, False), positions=i32(pos), base=1.0)  # one radian a position


def test_rope_given_frequencies(ops):
    """Frequencies of any size and sign, an even number of them zero."""
    c = TreeCase([(8, 8)], 2, 1, 64, "f16", "f32", seed=4)
    f = [(-1) ** i * 10.0 ** (i / 4 - 4) if i % 3 else 0.0 for i in range(32)]
    rope = ops.Rope(64, freq=f, device="cuda")
    pool, rows = c.ops()
    got = ops.rope_write(pool, rows, rope, c.q, c.new_k, c.new_v)
    want, b = turned(c.q[:8], list(range(8)), 64, torch.tensor(f, dtype=torch.double, device="cuda"), None, 0)
    assert_within(got[:8], want, rounded(b, want, torch.float32))


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dh", [64, 192, 256])
def test_rope_write_layouts(ops, kv, dh):
    """Slices of one projection's output, odd offsets, heads first, a broadcast row, in place, other outputs."""
    c = TreeCase([(9, 30), (4, 4)], 3, 1, dh, kv, "bf16", seed=5)
    qkv = torch.randn(c.n_rows, 5, dh, device="cuda").bfloat16()
    check_rope(ops, c, 64, q=qkv[:, :3], k=qkv[:, 3:4], v=qkv[:, 4:], parents=c.parents)
    odd = torch.randn(c.n_rows * 5 * dh + 1, device="cuda").bfloat16()[1:].view(c.n_rows, 5, dh)
    check_rope(ops, c, 64, q=odd[:, :3], k=odd[:, 3:4], v=odd[:, 4:])
    first = torch.randn(3, c.n_rows, dh, device="cuda").bfloat16().transpose(0, 1)
    check_rope(ops, c, 64, q=first, k=c.new_k[:1].expand(c.n_rows, 1, dh), v=c.new_v)
    q = c.q.clone()
    check_rope(ops, c, 64, q=q, out=q)  # in place
    wide = torch.zeros(c.n_rows, 3, dh + 3, device="cuda").bfloat16()
    wide[..., :dh] = c.q
    check_rope(ops, c, 64, out=wide[..., :dh])
    assert not wide[..., dh:].any()


def test_rope_write_rows_without_a_slot(ops):
    c = TreeCase([(20, 20), (6, 20)], 2, 1, 64, "f16", "f32", seed=6)
    c.tables[0, 0], c.tables[1, 1] = -1, c.n_pages
    check_rope(ops, c, 64, parents=c.parents)
    c = TreeCase([(5, 5)], 2, 1, 64, "q8", "f32", seed=7)
    c.kv_len[0] = 2
    c.seqs = [(5, 2)]
    check_rope(ops, c, 64)  # positions -3 .. 1
    check_rope(ops, c, 64, parents=c.parents)


def test_rope_norm_of_small_and_zero_heads(ops):
    """eps carries heads of zeros and of tiny values; a NaN stays in its own head."""
    c = TreeCase([(6, 6)], 2, 1, 128, "f16", "f32", seed=8, pad_rows=0)
    c.q[0] = 0
    c.q[1] *= 1e-6
    c.q[2] *= 1e-19
    c.q[3] *= 1e15
    c.q[4, 0, 5] = math.nan
    clean = c.q.clone()
    clean[4, 0] = 0
    gain = torch.ones(128, device="cuda")
    rope = ops.Rope(128, 1e7, gain, gain, EPS)
    pool, rows = c.ops()
    got = ops.rope_write(pool, rows, rope, c.q, c.new_k, c.new_v)
    assert bool(torch.isnan(got[4, 0]).all()) and not got[0].any()
    want, b = turned(clean, list(range(6)), 128, freqs(128), gain, EPS)
    keep = torch.ones(6, 2, dtype=torch.bool, device="cuda")
    keep[4, 0] = False
    assert_within(got[keep], want[keep], rounded(b, want, torch.float32)[keep])


@pytest.mark.parametrize("dh", [64, 192, 256])
def test_rope_norm_beyond_the_squares_of_32_bits(ops, dh):
    """Heads whose squares overflow, or with a small eps vanish, in 32 bits: normalised all the same."""
    c = TreeCase([(9, 9)], 2, 1, dh, "f16", "f32", seed=18, pad_rows=0)
    c.q[0] *= 1e19
    c.q[1] *= 1e37
    c.q[2, 1] = 3e38
    c.q[3] *= 1e-20
    c.q[4] *= 1e-36
    c.q[5, 0, 1:] = 0
    c.q[6, 0, 3], c.q[7, 1, 2] = math.inf, math.nan
    c.q[8] = 0
    clean = torch.where(torch.isfinite(c.q), c.q, torch.ones_like(c.q))
    for eps in (EPS, 1e-38, 0.0):
        gain = torch.rand(dh, device="cuda") + 0.5
        rope = ops.Rope(64, 1e4, gain, gain, eps)
        pool, rows = c.ops()
        got = ops.rope_write(pool, rows, rope, c.q, c.new_k, c.new_v)
        want, b = turned(clean, list(range(9)), 64, freqs(64, 1e4), gain, eps)
        keep = torch.ones(9, 2, dtype=torch.bool, device="cuda")
        keep[6, 0] = keep[7, 1] = keep[8] = False
        assert_within(got[keep], want[keep], rounded(b, want, torch.float32)[keep])
        assert bool(torch.isnan(got[6, 0]).any()) and bool(torch.isnan(got[7, 1]).all())
        assert bool(torch.isnan(got[8]).all()) if eps == 0 else not got[8].any()


def test_rope_write_many_rows(ops):
    """More rows than one head a group is for, an odd number of heads among the groups."""
    c = TreeCase([(700, 700), (333, 1200)], 7, 2, 256, "f16", "f16", seed=9, kind="chain")
    check_rope(ops, c, 192)
    c = TreeCase([(1900, 1900)], 9, 1, 64, "q8", "bf16", seed=10, kind="chain")
    check_rope(ops, c, 64, (True, True))


def test_rope_plain_write_agrees_with_kv_write(ops):
    """No dims turned and no gains: what kv_write stores, bit for bit."""
    for kv in ("f16", "q8"):
        c = TreeCase([(33, 50), (4, 4)], 2, 2, 128, kv, "f32", seed=11)
        pool, rows = c.ops()
        ops.kv_write(pool, rows, c.new_k, c.new_v)
        want = {n: t.clone() for n, t in c.pool.items()}
        for n in c.pool:
            c.pool[n].zero_()
            want[n][torch.isnan(want[n].float())] = 0
        ref = {n: torch.zeros_like(t) for n, t in c.pool.items()}
        d = TreeCase([(33, 50), (4, 4)], 2, 2, 128, kv, "f32", seed=11)
        d.pool = ref
        ops.kv_write(d.ops()[0], rows, c.new_k, c.new_v)
        q = ops.rope_write(pool, rows, ops.Rope(0, device="cuda"), c.q, c.new_k, c.new_v)
        assert torch.equal(q[:c.rows_used], c.q[:c.rows_used])
        for n in c.pool:
            assert torch.equal(bits(c.pool[n]), bits(ref[n])), n


# ------------------------------------------------------------ tree attention
def check_tree(ops, c, window=0, sinks=0, gate=False, **kw):
    pool, rows = c.ops()
    out = torch.full_like(c.q, 5.0)
    ops.attend(pool, rows, c.q, window=window, sinks=sinks, gate=c.gate if gate else None, out=out, parents=c.parents, **kw)
    want, bound = c.tree_ref(window, sinks, gate, scale=kw.get("scale"))
    assert_within(out[:c.rows_used], want, bound)
    assert bool((out[c.rows_used:] == 5.0).all())
    return out


TREES = [([(1, 1)], 1, 1, 64), ([(3, 3), (1, 16), (5, 17)], 4, 2, 64), ([(8, 135), (7, 128), (16, 129), (1, 400)], 6, 1, 128),
         ([(13, 700), (1, 1), (31, 31), (5, 260)], 6, 2, 192), ([(8, 4104)], 24, 4, 256), ([(16, 1000), (16, 77)], 24, 4, 256),
         ([(64, 300)], 32, 1, 64), ([(130, 130)], 1, 1, 128), ([(64, 515), (2, 2), (100, 100)], 12, 2, 256),
         ([(257, 600), (1, 3)], 8, 8, 128), ([(200, 333)], 5, 1, 192), ([(300, 2000), (0, 9), (43, 43)], 12, 2, 256),
         ([(90, 90)], 48, 1, 64), ([(2, 200)], 130, 1, 128), ([(3, 60)], 256, 1, 256)]


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("seqs,hq,hkv,dh", TREES)
def test_tree_attend(ops, seqs, hq, hkv, dh, dtype, kv):
    check_tree(ops, TreeCase(seqs, hq, hkv, dh, kv, dtype, seed=4))


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_tree_attend_shapes_of_trees(ops, kind, kv):
    check_tree(ops, TreeCase([(70, 200), (9, 9), (1, 130)], 6, 2, 128, kv, "f16", seed=5, kind=kind), gate=True)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (7, 4), (64, 0), (130, 140), (500, 1), (100000, 5)])
@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("kind", ["random", "chain"])
def test_tree_attend_windows(ops, window, sinks, kv, kind):
    c = TreeCase([(33, 700), (12, 12), (5, 300), (150, 160)], 4, 2, 64, kv, "f16", seed=6, kind=kind)
    check_tree(ops, c, window, sinks)


def test_a_chain_is_the_causal_attention(ops):
    """The same tokens are seen: equal but for the order in which blocks count as partly seen."""
    for seqs, window, sinks in (([(40, 400), (3, 3)], 0, 0), ([(140, 300)], 50, 4)):
        c = TreeCase(seqs, 6, 2, 128, "f16", "f16", seed=7, kind="chain")
        pool, rows = c.ops()
        a = ops.attend(pool, rows, c.q, window=window, sinks=sinks)
        b = check_tree(ops, c, window, sinks)
        u = c.rows_used
        _, bound = c.tree_ref(window, sinks)
        assert bool(((a[:u].double() - b[:u].double()).abs() <= 2 * bound).all())


def test_parents_that_are_none(ops):
    """Values that name no earlier node make a root, whatever they are."""
    par = [-1, 1, 7, -2 ** 31, 2 ** 31 - 1, 0, 4, 100]
    c = TreeCase([(8, 40)], 4, 2, 64, "f16", "f16", seed=8, parents=par)
    assert [len(x) for x in c.lines[0]] == [1, 1, 1, 1, 1, 2, 2, 1]
    check_tree(ops, c)
    check_tree(ops, c, 3, 1)


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_unseen_nodes_may_hold_anything(ops, kv):
    """Infinities and NaN in siblings' rows have no effect; a node's own lineage counts."""
    c = TreeCase([(24, 150), (9, 9)], 4, 2, 128, kv, "f16", seed=9)
    for i, (n, T) in enumerate(c.seqs):
        for j, bad in ((1, math.nan), (4, math.inf), (7, -math.inf), (n - 1, math.nan)):
            slot = T - n + j
            page = int(c.tables[i, slot // 16])
            if kv == "f16":
                c.pool["v"][page, :, slot % 16, ::7] = bad
            else:
                c.pool["v_scale"][page, :, slot % 16, 1] = bad
                c.pool["v"][page, :, slot % 16, 32:64] = 1 + torch.arange(32, device="cuda", dtype=torch.int8)
        # keys of the last node, which only it sees: scores of NaN would show in every other node
        page = int(c.tables[i, (T - 1) // 16])
        if kv == "f16":
            c.pool["k"][page, :, (T - 1) % 16] = math.nan
        else:
            c.pool["k_scale"][page, :, (T - 1) % 16] = math.nan
    for name in ("k", "v"):
        x = c.pool[name].double()
        c.value[name] = x if kv == "f16" else (x.unflatten(-1, (-1, 32)) * c.pool[name + "_scale"].double()[..., None]).flatten(-2)
    pool, rows = c.ops()
    out = ops.attend(pool, rows, c.q, parents=c.parents)
    own_key = [int(c.start[i + 1]) - 1 for i in range(2)]  # (these two rows have NaN scores)
    want, bound = c.tree_ref()
    keep = torch.ones(c.rows_used, dtype=torch.bool, device="cuda")
    keep[own_key] = False
    assert_within(out[:c.rows_used][keep], want[keep], bound[keep])
    assert not torch.isfinite(out[own_key]).any()


@pytest.mark.parametrize("seqs,hq,hkv,dh,kv", [([(64, 30000)], 24, 4, 256, "f16"), ([(64, 52000)], 24, 4, 256, "q8"), ([(100, 100000)], 8, 4, 64, "f16"),
                                               ([(45, 70001)], 12, 2, 192, "f16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5), (20000, 0)])
def test_tiles_that_share_a_far_context(ops, seqs, hq, hkv, dh, kv, window, sinks):
    """Contexts beyond the L2 cache, several tiles of one sequence: all tiles are cut at the same blocks, into more
    pieces than a narrow window has blocks."""
    c = TreeCase(seqs, hq, hkv, dh, kv, "f16", seed=19)
    check_tree(ops, c, window, sinks)
    if not window:
        from ops_helpers import Case
        pool, rows = c.ops()
        out = ops.attend(pool, rows, c.q)
        want, bound = Case.attend_ref(c)
        assert_within(out[:c.rows_used], want, bound)


def test_nodes_without_pages_or_slots(ops):
    c = TreeCase([(20, 150), (30, 40)], 4, 2, 64, "f16", "f16", seed=10)
    c.tables[0, 2], c.tables[0, 8], c.tables[1, 0], c.tables[1, 1] = -1, c.n_pages, -7, -1
    check_tree(ops, c)
    c = TreeCase([(12, 12)], 4, 2, 64, "f16", "f16", seed=11, kind="forest")
    c.kv_len[0] = 5
    c.seqs = [(12, 5)]
    out = check_tree(ops, c)
    assert not out[:7].any()  # rows at negative slots see nothing
    c = TreeCase([(6, 6)], 4, 2, 64, "q8", "bf16", seed=12)
    c.tables[:] = -1
    assert not check_tree(ops, c)[:6].any()


def test_large_values_of_a_q8_tree(ops):
    """Scales of 512 and more take the second pass; there the tree's mask holds too."""
    c = TreeCase([(20, 200), (3, 3)], 4, 2, 64, "q8", "f16", seed=13)
    page, slot = int(c.tables[0, 190 // 16]), 190 % 16
    c.pool["v_scale"][page, :, slot] = 600.0
    c.pool["v"][page, :, slot] = 1
    for name in ("k", "v"):
        c.value[name] = (c.pool[name].double().unflatten(-1, (-1, 32)) * c.pool[name + "_scale"].double()[..., None]).flatten(-2)
    pool, rows = c.ops()
    out = ops.attend(pool, rows, c.q, parents=c.parents)
    want, bound = c.tree_ref()
    # beside such a token small values are rounded 2^8 coarser (documented): T 2^-17 of the largest value on top
    assert_within(out[:c.rows_used], want, bound + 200 * 2.0 ** -17 * 600)
    far = torch.tensor([190 - 180 not in line for line in c.lines[0]], device="cuda")
    plain = want[:20][far]
    assert bool(((out[:20][far].double() - plain).abs() <= bound[:20][far] + 200 * 2.0 ** -17 * 4).all())


# ---------------------------------------------------------------- acceptance
def accept_case(seqs, vocab, dtype, seed=0, agree=0.8, pad=2, parents=None):
    g = torch.Generator().manual_seed(seed)
    rows = sum(seqs)
    par = random_parents([(q, q) for q in seqs], seed) if parents is None else parents
    tok = torch.randint(0, vocab, (rows + pad,), generator=g)
    x = torch.randn(rows + pad, vocab, generator=g)
    at = 0
    for q in seqs:
        for j in range(1, q):
            if par[at + j] >= 0 and float(torch.rand(1, generator=g)) < agree:
                x[at + par[at + j], tok[at + j]] = 6 + float(torch.rand(1, generator=g))
        at += q
    return par, tok.to(torch.int32).cuda(), x.to(dtype).cuda()


def check_accept(ops, seqs, par, tok, logits, pass_parents=True):
    start = np.concatenate([[0], np.cumsum(seqs)]).astype(np.int32).tolist()
    n = logits.shape[0]
    rows = ops.KVRows(i32(start), i32([0] * len(seqs)), torch.zeros(len(seqs), 1, dtype=torch.int32, device="cuda"), n)
    p = i32(list(par) + [0] * (n - len(par))) if pass_parents else None
    path, count, emitted = ops.tree_accept(rows, p, tok, logits)
    assert path.dtype == count.dtype == emitted.dtype == torch.int32
    host, tl = logits.float().cpu().tolist(), tok.tolist()
    longest = 0
    for i, q in enumerate(seqs):
        a, b = start[i], start[i + 1]
        want, out = walk(list(par[a:b]), tl[a:b], host[a:b]) if q else ([], [])
        assert int(count[i]) == len(want)
        assert path[a:b].tolist() == want + [-1] * (q - len(want))
        assert emitted[a:b].tolist() == out + [-1] * (q - len(want))
        longest = max(longest, len(want))
    return longest


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("seqs,vocab", [([1], 1), ([1, 8, 3], 7), ([8], 2048), ([16, 16, 0, 5], 2047), ([40], 2049), ([300, 33], 100),
                                        ([12], 70001), ([3, 1], 248320)])
def test_tree_accept(ops, seqs, vocab, dtype):
    longest = check_accept(ops, seqs, *accept_case(seqs, vocab, dtype, seed=len(seqs) + vocab))
    assert longest >= 1


def test_long_paths_and_chains(ops):
    q = 200
    par, tok, x = accept_case([q], 50, torch.float32, 3, agree=1.0, parents=[j - 1 for j in range(q)], pad=0)
    x[:] = 0
    for j in range(1, q):
        x[j - 1, tok[j]] = 1
    assert check_accept(ops, [q], par, tok, x) == q
    assert check_accept(ops, [q], par, tok, x, pass_parents=False) == q
    x[77, tok[78]] = -1
    assert check_accept(ops, [q], par, tok, x, pass_parents=False) == 78


def test_ties_zeros_infinities_and_nan(ops):
    seqs, par = [4, 3, 3, 2, 2, 3], [-1, 0, 0, 1, -1, 0, 1, -1, 0, 0, -1, 0, -1, 0, -1, 0, 1]
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.full((17, 5000), -2.0)
        tok = torch.zeros(17, dtype=torch.int32)
        x[0, [4999, 1234, 2600]] = 3.0      # the lowest index of equal ones, across parts of a row
        tok[1], tok[2] = 1234, 1234         # two children that agree: the lower one
        x[4, :] = -math.inf                 # all equal
        tok[5] = 0
        x[7, 17], x[7, 3] = math.nan, math.inf  # a NaN: nothing is accepted
        tok[8], tok[9] = 3, -1
        x[10, :], x[10, 4000], x[10, 40] = -5.0, -0.0, 0.0  # -0 and 0 are equal
        tok[11] = 40
        x[12, 77] = math.inf
        tok[13] = 77
        x[14, :] = -math.inf
        x[14, 4321] = torch.finfo(dtype).min
        tok[15] = 4321
        x[15, 4999] = 1.0
        tok[16] = 4999
        got = check_accept(ops, seqs, par, tok.cuda(), x.to(dtype).cuda())
        assert got == 3


def test_accept_roots_and_bad_parents(ops):
    """Nodes whose parent is no earlier one are no children; the first row stands whatever its parent says."""
    x = torch.zeros(6, 10, device="cuda")
    x[:, 3] = 1
    tok = i32([3] * 6)
    assert check_accept(ops, [6], [5, -1, 2, 9, 0, 4], tok, x) == 3  # 0, 4, 5


def test_accept_layouts(ops):
    """Rows further apart than the vocabulary, odd offsets, more rows than the tree's."""
    seqs = [9, 20]
    par, tok, x = accept_case(seqs, 1000, torch.float32, 5)
    check_accept(ops, seqs, par, tok, x)
    for pad, skip in ((5, 0), (8, 3), (24, 8)):
        wide = torch.full((x.shape[0], 1000 + pad), 99.0, device="cuda")
        wide[:, skip:] = 99.0
        view = wide.flatten()[skip if skip < pad else 0:]
        view = wide.as_strided((x.shape[0], 1000), (1000 + pad, 1), min(skip, pad))
        view.copy_(x)
        check_accept(ops, seqs, par, tok, view)
        half = torch.full((x.shape[0], 1000 + pad), 99.0, device="cuda", dtype=torch.float16)
        hv = half.as_strided((x.shape[0], 1000), (1000 + pad, 1), min(skip, pad))
        hv.copy_(x)
        check_accept(ops, seqs, par, tok, hv)


def test_accept_of_no_rows(ops):
    rows = ops.KVRows(i32([0, 0, 0]), i32([4, 4]), torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 0)
    path, count, emitted = ops.tree_accept(rows, i32([]), i32([]), torch.zeros(0, 5, device="cuda"))
    assert count.tolist() == [0, 0] and path.numel() == emitted.numel() == 0


# ---------------------------------------------------------- kept and copied
def layered(n_layers, n_pages, hkv, dh, kv, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n_layers, n_pages, hkv, 16, dh)
    out = {}
    for n in ("k", "v"):
        if kv == "f16":
            out[n] = torch.randint(-32768, 32767, shape, generator=g, device="cuda", dtype=torch.int16)
        else:
            out[n] = torch.randint(-128, 127, shape, generator=g, device="cuda", dtype=torch.int8)
            out[n + "_scale"] = torch.randint(-32768, 32767, shape[:-1] + (dh // 32,), generator=g, device="cuda", dtype=torch.int16)
    return out


def as_layers(ops, pool):
    return ops.KVLayers(pool["k"], pool["v"], pool.get("k_scale"), pool.get("v_scale"))


def kept_entries(keep, q):
    """The entries that count, by the documented rule."""
    out = []
    for k in keep:
        if not (out[-1] if out else -1) < k < q:
            break
        out.append(k)
    return out


def check_keep(ops, n_layers, hkv, dh, kv, seqs, keeps, tables=None, kv_len=None, pool=None, seed=0):
    pages = [-(-T // 16) for _, T in seqs]
    n_pages = sum(pages) + 2
    if tables is None:
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        width, at, tables = max(pages + [1]) + 1, 0, []
        for n in pages:
            tables.append(order[at:at + n] + [-1] * (width - n))
            at += n
    pool = layered(n_layers, n_pages, hkv, dh, kv, seed) if pool is None else pool
    want = {n: t.clone() for n, t in pool.items()}
    start, entries, lengths = [0], [], []
    for i, ((q, T), keep) in enumerate(zip(seqs, keeps)):
        T = kv_len[i] if kv_len else T
        start.append(start[-1] + q)
        entries += list(keep) + [-1] * (q - len(keep))
        good, base = kept_entries(keep, q), T - q
        lengths.append(max(0, base + len(good)))
        place = lambda s: (tables[i][s // 16], s % 16) if 0 <= s < 16 * len(tables[i]) and 0 <= tables[i][s // 16] < n_pages else None  # noqa: E731
        pairs = [(place(base + k), place(base + t)) for t, k in enumerate(good)]
        pairs = [(a, b) for a, b in pairs if a and b and a != b]
        if pairs:
            (sp, ss), (dp, ds) = (torch.tensor(x, device="cuda").T for x in zip(*pairs))
            for n in want:
                want[n][:, dp, :, ds] = pool[n][:, sp, :, ss]  # (the pool before the call)
    rows = ops.KVRows(i32(start), i32(kv_len or [T for _, T in seqs]), i32(tables), len(entries))
    got = ops.kv_keep(as_layers(ops, pool), rows, i32(entries))
    assert got.tolist() == lengths
    for n in want:
        assert torch.equal(pool[n], want[n]), n


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("n_layers,hkv,dh", [(1, 1, 64), (3, 2, 128), (2, 3, 192), (17, 4, 256)])
def test_keep_accepted_paths(ops, n_layers, hkv, dh, kv):
    check_keep(ops, n_layers, hkv, dh, kv, [(16, 40), (1, 1), (8, 8), (5, 100), (0, 7)], [[0, 2, 3, 9, 15], [0], [1, 2, 3], [], []])
    check_keep(ops, n_layers, hkv, dh, kv, [(64, 200)], [list(range(64))])  # nothing moves
    check_keep(ops, n_layers, hkv, dh, kv, [(64, 200)], [list(range(1, 64))])  # everything moves by one


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("shift", [1, 7, 127, 128, 129, 1000])
def test_keep_long_contexts_in_place(ops, kv, shift):
    """What moves overlaps where it goes, over many tokens at a time."""
    n = 3000
    check_keep(ops, 2, 2, 64 if shift % 2 else 256, kv, [(n, n), (n // 3, n // 2)],
               [[0, 1] + list(range(2 + shift, n)), list(range(0, n // 3, 2))])
    g = torch.Generator().manual_seed(shift)
    some = (torch.rand(n, generator=g) < 0.7).nonzero()[:, 0].tolist()
    check_keep(ops, 1, 1, 128, kv, [(n, n)], [some], seed=shift)


def test_keep_lists_that_end_early(ops):
    for keep in ([3, 2, 5], [0, 4, 4, 6], [0, 16], [0, 2 ** 31 - 1, 3], [-5, 1], [-1], [2, -2 ** 31, 4]):
        check_keep(ops, 2, 1, 64, "f16", [(16, 40), (4, 9)], [keep, [1, 3]])
    check_keep(ops, 1, 1, 64, "f16", [(400, 400)], [list(range(5, 140)) + [7] + list(range(150, 300))])


def test_keep_without_pages_or_slots(ops):
    tables = [[0, -1, 2, 99, 4], [3, 1, -5, -1, -1]]
    check_keep(ops, 2, 2, 64, "q8", [(60, 70), (20, 30)], [list(range(3, 60)), list(range(0, 20, 3))], tables=tables)
    check_keep(ops, 1, 1, 64, "f16", [(12, 16)], [[2, 5, 9, 11]], kv_len=[6])  # slots -6 .. 5


def test_layers_of_a_larger_pool(ops):
    """Every other layer of a pool, and one of its middle layers: the others keep their bytes."""
    for kv in ("f16", "q8"):
        whole = layered(6, 6, 2, 64, kv, 3)
        before = {n: t.clone() for n, t in whole.items()}
        check_keep(ops, 3, 2, 64, kv, [(16, 40)], [[2, 5, 6]], tables=[[1, 4, 0]], pool={n: t[1::2] for n, t in whole.items()})
        for n in whole:
            assert torch.equal(whole[n][::2], before[n][::2]) and not torch.equal(whole[n], before[n])
        part = {n: t[2:3] for n, t in whole.items()}
        want = {n: t.clone() for n, t in whole.items()}
        for n in want:
            want[n][2, 5] = want[n][2, 0]
        ops.kv_copy(as_layers(ops, part), i32([0]), i32([5]))
        for n in whole:
            assert torch.equal(whole[n], want[n]), n


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("n_layers,hkv,dh,n_pages", [(1, 1, 64, 9), (17, 4, 256, 20), (2, 3, 192, 300), (3, 8, 128, 70)])
def test_copy(ops, n_layers, hkv, dh, n_pages, kv):
    pool = layered(n_layers, n_pages, hkv, dh, kv, 4)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).tolist()
    half = n_pages // 2
    src, dst = order[:half], order[half:2 * half]
    src[1] = src[0]  # one page several times
    extra = ([-1, 0, n_pages, 2 ** 31 - 1, src[0]], [dst[0], -1, dst[0], dst[0], n_pages])  # passed over
    want = {n: t.clone() for n, t in pool.items()}
    for n in want:
        want[n][:, dst] = want[n][:, src]
    ops.kv_copy(as_layers(ops, pool), i32(src + extra[0]), i32(dst + extra[1]))
    for n in want:
        assert torch.equal(pool[n], want[n]), n
    ops.kv_copy(as_layers(ops, pool), i32([]), i32([]))


def test_copy_more_pairs_than_a_grid_has_rows(ops):
    pool = layered(1, 140001, 1, 64, "f16", 5)
    want = {n: t.clone() for n, t in pool.items()}
    src, dst = torch.arange(70000, device="cuda"), 70000 + torch.randperm(70000, device="cuda")
    for n in want:
        want[n][:, dst] = want[n][:, src]
    ops.kv_copy(as_layers(ops, pool), src.int(), dst.int())
    for n in want:
        assert torch.equal(pool[n], want[n])


def test_offsets_beyond_32_bits(ops):
    """Layers more than 2^32 bytes apart."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    pool = {n: torch.zeros(3, 90000, 2, 16, 256, dtype=torch.int16, device="cuda") for n in ("k", "v")}
    for n, t in pool.items():
        t[:, 89999] = torch.arange(3, device="cuda", dtype=torch.int16)[:, None, None, None] + (5 if n == "k" else 9)
    ops.kv_copy(as_layers(ops, pool), i32([89999]), i32([89990]))
    rows = ops.KVRows(i32([0, 8]), i32([24]), i32([[89998, 89999]]), 8)
    ops.kv_keep(as_layers(ops, pool), rows, i32([6, 7, -1, 0, 0, 0, 0, 0]))
    for n, t in pool.items():
        for i in range(3):
            x = i + (5 if n == "k" else 9)
            assert bool((t[i, 89990] == x).all()) and bool((t[i, 89999] == x).all())
            assert int(t[i].ne(0).sum()) == 2 * 2 * 16 * 256
        t.zero_()


# ------------------------------------------------------------------ together
class Flow:
    """A layer's step over trees: rotate and write, attend, verify, keep."""

    def __init__(self, ops, kv, seqs, seed=0, hq=6, hkv=2, dh=128, vocab=3000):
        self.ops, self.vocab = ops, vocab
        self.c = TreeCase(seqs, hq, hkv, dh, kv, "f16", seed=seed, pad_rows=0)
        c = self.c
        for n in c.pool:
            c.pool[n].nan_to_num_(0) if c.pool[n].is_floating_point() else None
        gain = torch.rand(dh, device="cuda") + 0.5
        self.rope = ops.Rope(64, 1e4, gain, gain, EPS)
        self.proj = torch.randn(hq * dh, vocab, device="cuda", dtype=torch.float16) / math.sqrt(hq * dh)
        self.qkv = torch.randn(c.n_rows, hq + 2 * hkv, dh, device="cuda", dtype=torch.float16)
        self.tokens = torch.randint(0, vocab, (c.n_rows,), device="cuda", dtype=torch.int32)
        self.hq, self.hkv = hq, hkv
        self.layers = ops.KVLayers(*(None if c.pool.get(n) is None else c.pool[n][None] for n in ("k", "v", "k_scale", "v_scale")))

    def verify(self):
        ops, c = self.ops, self.c
        pool, rows = c.ops()
        q, k, v = self.qkv.split([self.hq, self.hkv, self.hkv], 1)
        q = ops.rope_write(pool, rows, self.rope, q, k, v, parents=c.parents)
        o = ops.attend(pool, rows, q, parents=c.parents)
        return q, o, o.flatten(1) @ self.proj

    def step(self):
        q, o, logits = self.verify()
        path, count, emitted = self.ops.tree_accept(self.c.ops()[1], self.c.parents, self.tokens, logits)
        kv_len = self.ops.kv_keep(self.layers, self.c.ops()[1], path)
        return q, o, logits, path, count, emitted, kv_len


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_a_step_over_trees(ops, kv):
    """The accepted path of a tree leaves the cache as a chain of those tokens would have, and its nodes' attention
    is that chain's."""
    f = Flow(ops, kv, [(16, 200), (7, 7), (30, 65)], seed=1)
    c = f.c
    _, _, logits = f.verify()
    # drafts that agree with the model along some line of each tree
    at, paths = 0, []
    for i, (q, T) in enumerate(c.seqs):
        line = max(c.lines[i], key=len)
        line = line if line[0] == 0 else [0]
        for a, b in zip(line, line[1:]):
            f.tokens[at + b] = logits[at + a].float().argmax().int()
        paths.append(line)
        at += q
    _, o, logits, path, count, emitted, kv_len = f.step()
    host, tl, at = logits.float().cpu().tolist(), f.tokens.tolist(), 0
    chain = Flow(ops, kv, c.seqs, seed=1)
    d = chain.c
    for n in d.pool:
        d.pool[n].copy_(c.pool[n])
    rows_of, start, lens = [], [0], []
    for i, (q, T) in enumerate(c.seqs):
        want, out = walk([x if x < j else -1 for j, x in enumerate(c.parent_list[at:at + q])], tl[at:at + q], host[at:at + q])
        assert want[:len(paths[i])] == paths[i] or len(want) >= len(paths[i])
        n = int(count[i])
        assert path[at:at + n].tolist() == want and emitted[at:at + n].tolist() == out
        assert int(kv_len[i]) == T - q + n
        rows_of += [at + x for x in want]
        start.append(start[-1] + n)
        lens.append(T - q + n)
        at += q
    # the same tokens as a chain over the kept cache
    pool, _ = d.ops()
    rows = ops.KVRows(i32(start), i32(lens), c.tables, len(rows_of))
    kept_k, kept_v = ops.kv_read(c.ops()[0], rows, torch.float32)
    sel = f.qkv[rows_of]
    q, k, v = sel.split([f.hq, f.hkv, f.hkv], 1)
    q = ops.rope_write(pool, rows, f.rope, q, k, v)
    got_k, got_v = ops.kv_read(pool, rows, torch.float32)
    assert torch.equal(kept_k, got_k) and torch.equal(kept_v, got_v)  # the same positions, so the same angles
    o2 = ops.attend(pool, rows, q)
    # each is within the attention's bound of the same exact value
    c2 = TreeCase([(b - a, n) for a, b, n in zip(start, start[1:], lens)], f.hq, f.hkv, c.dh, kv, "f16", pad_rows=0, kind="chain")
    c2.tables, c2.n_pages, c2.pool, c2.q = c.tables, c.n_pages, d.pool, q
    for name in ("k", "v"):
        x = d.pool[name].double()
        c2.value[name] = x if kv == "f16" else (x.unflatten(-1, (-1, 32)) * d.pool[name + "_scale"].double()[..., None]).flatten(-2)
    want, bound = c2.tree_ref()
    assert_within(o2, want, bound)
    assert_within(o[rows_of], want, bound)


def test_captured_steps(ops):
    """Two graphs of whole steps, replayed in turn with other inputs, give what eager calls give."""
    flows = [Flow(ops, kv, [(16, 200), (7, 30)], seed=s) for s, kv in ((2, "f16"), (3, "q8"))]
    pools = [{n: t.clone() for n, t in f.c.pool.items()} for f in flows]

    def reset(i):
        for n, t in pools[i].items():
            flows[i].c.pool[n].copy_(t)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in flows:
            f.step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for i, f in enumerate(flows):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f.step())
        graphs.append(g)
    for turn in range(3):
        for i, f in enumerate(flows):
            f.qkv.copy_(torch.randn_like(f.qkv))
            f.c.parents.copy_(i32(random_parents(f.c.seqs, 50 + turn)))
            f.tokens.copy_(torch.randint(0, f.vocab, f.tokens.shape, device="cuda", dtype=torch.int32))
            reset(i)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        after = [{n: t.clone() for n, t in f.c.pool.items()} for f in flows]
        for i, f in enumerate(flows):
            reset(i)
            for a, b in zip(got[i], f.step()):
                assert torch.equal(bits(a), bits(b))
            for n, t in after[i].items():
                assert torch.equal(bits(t), bits(f.c.pool[n])), n


def test_other_streams(ops):
    """Calls go to the current stream, behind what is queued there, two of them at once."""
    flows = [Flow(ops, "f16", [(16, 500)], seed=s) for s in (4, 5)]
    want = []
    for f in flows:
        keep = {n: t.clone() for n, t in f.c.pool.items()}
        want.append([t.clone() for t in f.step()])
        for n, t in keep.items():
            f.c.pool[n].copy_(t)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in flows], []
    for f, s in zip(flows, streams):
        qkv = f.qkv.clone()
        f.qkv.zero_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2000000)
            f.qkv.copy_(qkv)
            got.append(f.step())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(bits(x), bits(y))


# ------------------------------------------------------------------ an engine
@pytest.fixture(scope="module")
def engine_parts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gen import configs, synth
    model = dict(configs.TINY)
    return model, synth.make_weights(model, 0)


@pytest.mark.parametrize("q8", [0, 1])
def test_engine_clone_and_keep(engine_parts, q8):
    from speculative_decode_persistent_gb300 import mk
    model, weights = engine_parts
    eng = mk.Engine(model, weights, q8, 64)
    n = 70
    k, v = (torch.randn(1, n, model["hkv"], model["dh"], device="cuda").half() for _ in "kv")
    S = torch.randn(eng.state_views()[0].shape[2:], device="cuda")
    conv = torch.randn(eng.state_views()[1].shape[2:], device="cuda")
    eng.seq_load(2, k, v, S, conv)
    k0, v0 = eng.seq_kv(2, torch.float32)
    eng.clone_sequence(2, 5)
    a, b = eng.seq_get(2), eng.seq_get(5)
    assert b["length"] == n and not set(a["pages"].tolist()) & set(b["pages"].tolist())
    for x, y in zip(eng.seq_kv(5, torch.float32), (k0, v0)):
        assert torch.equal(x, y)
    assert torch.equal(b["S"], S) and torch.equal(b["conv"], conv)
    # the last 20 tokens were a tree; five of its nodes stay
    assert eng.seq_keep(5, 20, [0, 1, 4, 9, 19]) == 55
    kept = list(range(50)) + [50, 51, 54, 59, 69]
    for x, y in zip(eng.seq_kv(5, torch.float32), (k0, v0)):
        assert torch.equal(x, y[:, kept])
    for x, y in zip(eng.seq_kv(2, torch.float32), (k0, v0)):
        assert torch.equal(x, y)
    b = eng.seq_get(5)
    assert b["length"] == 55 and len(b["pages"]) == 4 and torch.equal(b["S"], S)
    eng.clone_sequence(5, 5)
    assert eng.seq_get(5)["length"] == 55
    for x, y in zip(eng.seq_kv(5, torch.float32), (k0, v0)):
        assert torch.equal(x, y[:, kept])
    for new_rows, keep in ((56, []), (5, [1, 1]), (5, [2, 1]), (5, [5]), (5, [-1]), (-1, [])):
        with pytest.raises(mk.MkError):
            eng.seq_keep(5, new_rows, keep)
    assert eng.seq_keep(5, 0, []) == 55 and eng.seq_keep(5, 55, []) == 0
    assert len(eng.seq_get(5)["pages"]) == 0


def test_engine_attends_to_a_tree(engine_parts):
    from speculative_decode_persistent_gb300 import mk
    model, weights = engine_parts
    eng = mk.Engine(model, weights, 0, 64)
    n, q = 90, 12
    k, v = (torch.randn(1, n, model["hkv"], model["dh"], device="cuda").half() for _ in "kv")
    eng.seq_load(0, k, v)
    c = TreeCase([(q, n)], model["hq"], model["hkv"], model["dh"], "f16", "f16", seed=3, pad_rows=0)
    info = eng.seq_get(0)
    c.tables, c.n_pages = i32([info["pages"].tolist()]), 64
    views = eng.kv_views()
    for name in ("k", "v"):
        c.value[name] = views[name][0].view(torch.float16).double()
    out = eng.attend(0, c.q, [0], [q], parents=c.parents)
    want, bound = c.tree_ref()
    assert_within(out, want, bound)
