"""Calls of the operators on trees that their documentation allows: as many sequences as a call may have, results
written over the queries or the gate, hints of any value, inputs from another stream, eager and captured."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import Case, assert_within  # noqa: E402
from tree_helpers import TreeCase  # noqa: E402
from test_gpu_tree_ops import accept_case, check_accept, check_keep, check_rope  # noqa: E402


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def bits(t):
    return t.view(torch.int16) if t.dtype in (torch.float16, torch.bfloat16) else t


def many(n, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 7, (n,), generator=g).tolist()
    return [(x, x + int(t)) for x, t in zip(q, torch.randint(0, 60, (n,), generator=g))]


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("n", [33, 1024])
def test_as_many_sequences_as_a_call_may_have(ops, n, kv):
    """Empty ones among them."""
    seqs = many(n, n)
    c = TreeCase(seqs, 4, 2, 64, kv, "f16", seed=n)
    check_rope(ops, c, 64, parents=c.parents)
    c = TreeCase(seqs, 4, 2, 64, kv, "f16", seed=n + 1)
    pool, rows = c.ops()
    for window, sinks in ((0, 0), (20, 2)):
        out = torch.full_like(c.q, 5.0)
        ops.attend(pool, rows, c.q, window=window, sinks=sinks, out=out, parents=c.parents)
        want, bound = c.tree_ref(window, sinks)
        assert_within(out[:c.rows_used], want, bound)
        assert bool((out[c.rows_used:] == 5.0).all())
    q = [a for a, _ in seqs]
    for vocab in (40, 5000):
        check_accept(ops, q, *accept_case(q, vocab, torch.float32, seed=n))
    keeps = [[j for j in range(a) if (j * 7 + s) % 3] for s, a in enumerate(q)]
    check_keep(ops, 2, 2, 64, kv, [(a, max(t, 1)) for a, t in seqs], keeps)


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("seqs,hq,hkv,dh", [([(8, 4104)], 24, 4, 256), ([(64, 515), (2, 2), (100, 100)], 12, 2, 256), ([(70, 200), (9, 9)], 6, 2, 192),
                                            ([(64, 30000)], 24, 4, 256)])
def test_trees_in_place(ops, seqs, hq, hkv, dh, kv):
    """Results over the queries, or over the gate."""
    c = TreeCase(seqs, hq, hkv, dh, kv, "bf16", seed=3)
    pool, rows = c.ops()
    u = c.rows_used
    want = ops.attend(pool, rows, c.q, gate=c.gate, parents=c.parents)[:u].clone()
    for over in ("q", "gate"):
        q, gate = c.q.clone(), c.gate.clone()
        t = q if over == "q" else gate
        behind = t[u:].clone()
        assert ops.attend(pool, rows, q, gate=gate, out=t, parents=c.parents) is t
        assert torch.equal(bits(t[:u]), bits(want)) and torch.equal(bits(t[u:]), bits(behind))


def test_large_q8_values_in_place(ops):
    """The second pass of large values reads the queries again: they are still there where the result replaces them."""
    c = TreeCase([(20, 900), (150, 400)], 12, 2, 128, "q8", "f16", seed=13)
    for page in (int(c.tables[0, 3]), int(c.tables[1, 20])):
        c.pool["v_scale"][page] = 600.0
        c.pool["v"][page] = 1
    pool, rows = c.ops()
    for parents in (c.parents, None):
        want = ops.attend(pool, rows, c.q, parents=parents)
        q = c.q.clone()
        ops.attend(pool, rows, q, out=q, parents=parents)
        assert torch.equal(bits(q[:c.rows_used]), bits(want[:c.rows_used]))


@pytest.mark.parametrize("hint", [0, 1, 40, 2 ** 31 - 1, None])
def test_any_hint(ops, hint):
    """max_q chooses kernels, never the result."""
    seqs = [(300, 700), (3, 20), (0, 5), (40, 40)]
    for kv in ("f16", "q8"):
        c = TreeCase(seqs, 6, 2, 128, kv, "f16", seed=8)
        pool, _ = c.ops()
        rows = ops.KVRows(c.start, c.kv_len, c.tables, c.n_rows, hint)
        want, bound = c.tree_ref()
        assert_within(ops.attend(pool, rows, c.q, parents=c.parents)[:c.rows_used], want, bound)
        want, bound = Case.attend_ref(c)
        assert_within(ops.attend(pool, rows, c.q)[:c.rows_used], want, bound)
    g = torch.Generator().manual_seed(1)
    tok = torch.randint(0, 9, (c.n_rows,), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(c.n_rows, 2500, generator=g).cuda()
    base = ops.KVRows(c.start, c.kv_len, c.tables, c.n_rows, 300)
    for a, b in zip(ops.tree_accept(base, c.parents, tok, x), ops.tree_accept(rows, c.parents, tok, x)):
        a, b = (t[:c.rows_used] if t.shape[0] == c.n_rows else t for t in (a, b))
        assert torch.equal(a, b)


class Forked:
    """Queries and rows made on one stream, rotated and written on a second, attended to on the first again."""

    def __init__(self, ops, kv, seed):
        self.ops = ops
        c = self.c = TreeCase([(16, 400), (7, 7)], 6, 2, 128, kv, "f16", seed=seed, pad_rows=0)
        for t in c.pool.values():
            if t.is_floating_point():
                t.nan_to_num_(0)
        self.rope = ops.Rope(64, 1e4, device="cuda")
        self.src = torch.randn(c.n_rows, 10, 128, device="cuda", dtype=torch.float16)
        self.qkv, self.spin = torch.empty_like(self.src), torch.zeros(1 << 24, device="cuda")
        self.other = torch.cuda.Stream()

    def run(self):
        """Each stream is given its work while what it waits for is still far from done."""
        ops, c = self.ops, self.c
        main = torch.cuda.current_stream()
        pool, rows = c.ops()
        for _ in range(4):
            self.spin.add_(1.0)
        torch.mul(self.src, 2.0, out=self.qkv)
        q, k, v = self.qkv.split([6, 2, 2], 1)
        self.other.wait_stream(main)
        with torch.cuda.stream(self.other):
            q = ops.rope_write(pool, rows, self.rope, q, k, v, parents=c.parents)
            for _ in range(4):
                self.spin.mul_(0.5)
            q2 = torch.mul(q, 0.5)
        main.wait_stream(self.other)
        o = ops.attend(pool, rows, q2, parents=c.parents)
        kk, vv = ops.kv_read(pool, rows)
        return q, o, kk, vv

    def want(self):
        ops, c = self.ops, self.c
        pool, rows = c.ops()
        q, k, v = (self.src * 2.0).split([6, 2, 2], 1)
        torch.cuda.synchronize()
        q = ops.rope_write(pool, rows, self.rope, q, k, v, parents=c.parents)
        torch.cuda.synchronize()
        q2 = q * 0.5
        torch.cuda.synchronize()
        o = ops.attend(pool, rows, q2, parents=c.parents)
        torch.cuda.synchronize()
        return [t.clone() for t in (q, o, *ops.kv_read(pool, rows))]


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_inputs_from_another_stream(ops, kv):
    f = Forked(ops, kv, 5)
    for turn in range(8):
        f.src.normal_()
        want = f.want()
        f.qkv.zero_()
        torch.cuda.synchronize()
        got = f.run()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(bits(a), bits(b)), turn


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_a_captured_fork(ops, kv):
    """The same captured: kernels behind kernels of another branch, and behind two at once."""
    f = Forked(ops, kv, 6)
    f.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f.run()
    for turn in range(8):
        f.src.normal_()
        want = f.want()
        f.qkv.zero_()
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(bits(a), bits(b)), turn
