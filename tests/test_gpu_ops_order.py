"""Pool operators one right behind the other: what a call reads was written by the kernel before it in the
stream, which may still be running when the call's own kernel starts. Every input of every call comes from a kernel
queued just before it, and the results are those of the same calls with a wait for the GPU between them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import Case  # noqa: E402
from tree_helpers import TreeCase  # noqa: E402


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def bits(t):
    return t.view(torch.int16) if t.dtype in (torch.float16, torch.bfloat16) else t


class Chain:
    """A layer's step over trees, every input made by a kernel right before the call that reads it."""

    def __init__(self, ops, kv, seqs, seed, hq=12, hkv=2, dh=128, vocab=700):
        self.ops, self.hq, self.hkv, self.dh = ops, hq, hkv, dh
        c = self.c = TreeCase(seqs, hq, hkv, dh, kv, "bf16", seed=seed, pad_rows=3)
        for t in c.pool.values():
            if t.is_floating_point():
                t.nan_to_num_(0)
        self.pool0 = {n: t.clone() for n, t in c.pool.items()}
        self.gain0 = torch.rand(dh, device="cuda") + 0.5
        self.gain = torch.empty_like(self.gain0)
        self.rope = ops.Rope(dh, 1e4, self.gain, self.gain)
        n = c.n_rows
        self.qkv = torch.empty(n, hq + 2 * hkv, dh, device="cuda", dtype=torch.bfloat16)
        self.proj = torch.randn(dh, vocab, device="cuda")
        self.src = {x: torch.empty_like(getattr(c, x)) for x in ("start", "kv_len", "tables", "parents")}
        for x, t in self.src.items():
            t.copy_(getattr(c, x))
        self.tokens, self.logits = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, vocab, device="cuda")
        self.layers = ops.KVLayers(*(None if c.pool.get(x) is None else c.pool[x][None] for x in ("k", "v", "k_scale", "v_scale")))
        self.pages = torch.empty(2, 3, dtype=torch.int32, device="cuda")

    def indexes(self, *names):
        """The call's rows, written anew by kernels, over zeros."""
        for x in names:
            t = getattr(self.c, x)
            t.fill_(0)
            torch.add(self.src[x], 0, out=t)

    def step(self, seed, wait):
        ops, c = self.ops, self.c
        out = []

        def done(*t):
            if wait:
                torch.cuda.synchronize()
            out.extend(x.clone() for x in t)
            if wait:
                torch.cuda.synchronize()

        g = torch.Generator(device="cuda").manual_seed(seed)
        fresh = torch.randn(self.qkv.shape, generator=g, device="cuda")
        token = torch.randint(0, self.logits.shape[1], self.tokens.shape, generator=g, device="cuda", dtype=torch.int32)
        for x, t in c.pool.items():
            t.copy_(self.pool0[x])
        self.gain.zero_()
        self.qkv.zero_()
        self.logits.zero_()
        torch.cuda.synchronize()
        pool, rows = c.ops()
        self.indexes("start", "kv_len", "tables", "parents")
        torch.mul(self.gain0, 1.25, out=self.gain)
        self.qkv.copy_(fresh * 2)
        q, k, v = self.qkv.split([self.hq, self.hkv, self.hkv], 1)
        assert ops.rope_write(pool, rows, self.rope, q, k, v, parents=c.parents, out=q) is q  # in place
        o = ops.attend(pool, rows, q, parents=c.parents)  # reads the rotated queries and the rows just written
        done(q, o)
        kk, vv = ops.kv_read(pool, rows, torch.float32)
        done(kk[:c.rows_used], vv[:c.rows_used])
        ops.kv_write(pool, rows, k, v)
        kk, vv = ops.kv_read(pool, rows, torch.float32)
        done(kk[:c.rows_used], vv[:c.rows_used])
        torch.matmul(o[:, 0].float(), self.proj, out=self.logits)
        torch.add(token, 0, out=self.tokens)
        path, count, emitted = ops.tree_accept(rows, c.parents, self.tokens, self.logits)
        lengths = ops.kv_keep(self.layers, rows, path)
        done(path[:c.rows_used], count, emitted[:c.rows_used], lengths, *c.pool.values())
        torch.add(torch.tensor([[0, 1, 2], [c.n_pages - 1, c.n_pages - 2, c.n_pages - 3]], dtype=torch.int32, device="cuda"), 0, out=self.pages)
        ops.kv_copy(self.layers, self.pages[0], self.pages[1])
        done(*c.pool.values())
        return out


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("seqs", [[(8, 300)], [(16, 2000), (5, 5), (30, 70)], [(200, 900), (64, 64)]])
def test_calls_right_behind_each_other(ops, kv, seqs):
    chain = Chain(ops, kv, seqs, seed=len(seqs))
    for turn in range(25):
        want, got = chain.step(turn, True), chain.step(turn, False)
        for i, (a, b) in enumerate(zip(want, got)):
            a, b = a[:chain.c.rows_used] if i < 2 else a, b[:chain.c.rows_used] if i < 2 else b
            assert torch.equal(torch.nan_to_num(bits(a)), torch.nan_to_num(bits(b))), (turn, i)


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("rows", [3, 40, 300])
def test_causal_calls_right_behind_each_other(ops, kv, rows):
    """The same for rows of a text: kv_write, then attend in place of its queries."""
    c = Case([(rows, 1500), (7, 90)], 12, 2, 256, kv, "bf16", seed=rows)
    pool, r = c.ops()
    q0, k0, v0 = c.q.clone(), c.new_k.clone(), c.new_v.clone()
    q, k, v = (torch.zeros_like(t) for t in (q0, k0, v0))

    def once(wait, f):
        for t in (q, k, v):
            t.zero_()
        torch.cuda.synchronize()
        for t, s in ((q, q0), (k, k0), (v, v0)):
            torch.mul(s, f, out=t)
        ops.kv_write(pool, r, k, v)
        if wait:
            torch.cuda.synchronize()
        return ops.attend(pool, r, q, out=q).clone()

    for turn in range(40):
        f = 1.0 + turn / 8
        assert torch.equal(bits(once(True, f)[:c.rows_used]), bits(once(False, f)[:c.rows_used])), turn


@pytest.mark.parametrize("seqs,hq,hkv,dh,kv", [([(8, 4104)], 24, 4, 256, "f16"), ([(16, 23016)] * 4, 24, 4, 256, "q8"),
                                               ([(64, 30064)], 24, 4, 256, "f16"), ([(1, 65), (13, 68), (37, 3001), (21, 21)], 4, 1, 64, "f16")])
def test_attention_repeats_itself(ops, seqs, hq, hkv, dh, kv):
    """The same inputs give the same bits, whatever ran in between and whatever the workspace held."""
    c = TreeCase(seqs, hq, hkv, dh, kv, "bf16", seed=5)
    pool, rows = c.ops()
    first = [ops.attend(pool, rows, c.q, parents=p) for p in (c.parents, None)]
    for turn in range(6):
        junk = torch.full((64 << 20,), float("nan"), device="cuda")
        del junk  # (its memory is what the next workspaces are cut from)
        c2 = TreeCase([(3, 50 + turn)], hq, hkv, dh, kv, "bf16", seed=turn)
        ops.attend(*c2.ops(), c2.q, parents=c2.parents)
        for p, want in zip((c.parents, None), first):
            got = ops.attend(pool, rows, c.q, parents=p)
            assert torch.equal(bits(got[:c.rows_used]), bits(want[:c.rows_used])), turn
