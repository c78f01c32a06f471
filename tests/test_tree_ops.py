"""Operators on trees of drafts, on the CPU: the C entries' refusals (all made
before any device work), the Python checks, the rotation's table, and the
references themselves on worked cases."""
import ctypes
import math
import os
import sys
from fractions import Fraction

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "tests"))
from test_ops import BAD_POOL, BAD_ROWS, _args, _pool, _rows  # noqa: E402


@pytest.fixture(scope="module")
def ops():
    from speculative_decode_persistent_gb300 import build as b
    b.build()
    from speculative_decode_persistent_gb300 import ops as o
    return o


def _rope(ops, **kw):
    d = ops.mk_dense(4096, 256, 64)
    a = ops.mk_rope_args(d, d, d, d, 4, 1, ops.mk_rope(4096, 4096, 4096, 64, 1e-6), None, None)
    for k, v in kw.items():
        if k in ("turns", "q_gain", "k_gain", "rot", "eps"):
            r = a.rope
            setattr(r, k, v)
            a.rope = r
        else:
            setattr(a, k, v)
    return a


def _tree(ops, **kw):
    t = ops.mk_tree_args(4096, 4096, 4096, 100000, 100000, 0, 4096, 4096, 4096, 4096, 1 << 30)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _layers(ops, n_layers=2, layer_stride=8 * 2 * 16 * 64, **kw):
    return ops.mk_kv_layers(_pool(ops, **kw), n_layers, layer_stride)


@pytest.mark.parametrize("pool_kw,rows_kw,status", [(p, {}, s) for p, s in BAD_POOL] + [({}, r, s) for r, s in BAD_ROWS])
def test_entries_refuse_bad_pools_and_rows(ops, pool_kw, rows_kw, status):
    p, r = _pool(ops, **pool_kw), _rows(ops, **rows_kw)
    assert ops.lib.mk_attend_tree(p, r, _args(ops), 4096, None) == status
    assert ops.lib.mk_rope_write(p, r, _rope(ops), None) == status
    assert ops.lib.mk_kv_keep(_layers(ops, 1, **pool_kw), r, 4096, None, None) == status
    if pool_kw:
        assert ops.lib.mk_kv_copy(_layers(ops, 1, **pool_kw), 4096, 4096, 1, None) == status
    else:
        assert ops.lib.mk_tree_accept(r, _tree(ops), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(rot=-64), -1), (dict(rot=128), -1), (dict(rot=32), -8),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(eps=math.inf), -1), (dict(turns=None), -1), (dict(turns=4100), -1),
    (dict(q_gain=4100), -1), (dict(k_gain=4104), -1), (dict(parents=4096, positions=4096), -1), (dict(hq=1 << 21), -8)])
def test_rope_write_refuses_bad_arguments(ops, kw, status):
    assert ops.lib.mk_rope_write(_pool(ops), _rows(ops), _rope(ops, **kw), None) == status


def test_rope_write_refuses_bad_tensors(ops):
    assert ops.lib.mk_rope_write(_pool(ops), _rows(ops), None, None) == -1
    for name in ("q", "out", "k", "v"):
        for at in (None, 4097):
            a = _rope(ops)
            setattr(a, name, ops.mk_dense(at, 256, 64))
            assert ops.lib.mk_rope_write(_pool(ops), _rows(ops), a, None) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=None), -1), (dict(logits=None), -1), (dict(logits=4098), -1), (dict(path=None), -1), (dict(count=None), -1),
    (dict(emitted=None), -1), (dict(vocab=0), -1), (dict(vocab=(1 << 30) + 1), -8), (dict(dtype=3), -1), (dict(work=None), -1),
    (dict(work=4100), -1), (dict(work_bytes=16), -1)])
def test_tree_accept_refuses_bad_arguments(ops, kw, status):
    assert ops.lib.mk_tree_accept(_rows(ops), _tree(ops, **kw), None) == status


def test_layers_and_lists_are_checked(ops):
    L = ops.lib
    assert L.mk_kv_copy(None, 4096, 4096, 1, None) == -1 and L.mk_kv_keep(None, _rows(ops), 4096, None, None) == -1
    for n, stride in ((0, 16384), (-1, 16384), (2, 16384 - 256), (2, 16384 + 64)):
        assert L.mk_kv_copy(_layers(ops, n, stride), 4096, 4096, 1, None) == -1
        assert L.mk_kv_keep(_layers(ops, n, stride), _rows(ops), 4096, None, None) == -1
    assert L.mk_kv_copy(_layers(ops, 65536), 4096, 4096, 1, None) == -8
    for src, dst, n in ((None, 4096, 1), (4096, None, 1), (4096, 4096, -1)):
        assert L.mk_kv_copy(_layers(ops), src, dst, n, None) == -1
    assert L.mk_kv_keep(_layers(ops), _rows(ops), None, 4096, None) == -1


def test_nothing_to_do_is_ok_without_a_device(ops):
    L, d = ops.lib, ops.mk_dense(None, 256, 64)
    assert L.mk_kv_copy(_layers(ops), None, None, 0, None) == 0
    assert L.mk_kv_keep(_layers(ops), _rows(ops, n_seqs=0), None, None, None) == 0
    assert L.mk_tree_accept(_rows(ops, n_seqs=0), _tree(ops, count=None), None) == 0
    for kw in (dict(n_seqs=0), dict(n_rows=0)):
        assert L.mk_rope_write(_pool(ops), _rows(ops, **kw), _rope(ops, q=d, out=d, k=d, v=d), None) == 0
        assert L.mk_attend_tree(_pool(ops), _rows(ops, **kw), _args(ops, q=d, out=d), 4096, None) == 0


def test_work_bytes(ops):
    w = lambda n, v, q: ops.lib.mk_tree_work_bytes(_rows(ops, n_rows=n, max_q=q), v)  # noqa: E731
    assert w(-1, 10, 1) == 0 and w(4, 0, 1) == 0 and w(4, (1 << 30) + 1, 1) == 0
    for n in (0, 1, 7, 64, 1000, 1 << 20):
        for v in (1, 2047, 2048, 2049, 248320, 1 << 30):
            for q in (1, 16, n):
                few = n <= 1024 and v <= 4096 and q * v <= 1 << 15  # one launch, nothing to keep between two
                parts = max(1, min(-(-v // 2048), max(1, -(-608 // max(n, 1))), 128))
                assert w(n, v, q) == 0 if few else w(n, v, q) >= n * (8 * parts + 4), (n, v, q)


# -------------------------------------------------------- the rotation's table
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068")


def _turns(ops, dims, base=1e7, freq=None):
    out = (ctypes.c_uint64 * max(dims // 2, 1))()
    f = None if freq is None else (ctypes.c_double * len(freq))(*freq)
    return ops.lib.mk_rope_turns(dims, base, f, out), list(out)[:dims // 2]


@pytest.mark.parametrize("dims,base", [(64, 1e7), (256, 1e4), (128, 5e5), (2, 1.0)])
def test_turns_are_the_frequencies(ops, dims, base):
    rc, t = _turns(ops, dims, base)
    assert rc == 0
    for i, x in enumerate(t):
        f = Fraction(base ** (-2.0 * i / dims)) / TWO_PI
        # pow and the quotient are doubles: two roundings of a value below 1/6 turn, the last bits of 2^64 fall away
        assert abs(Fraction(x, 1 << 64) - f) <= f * Fraction(1, 1 << 51) + Fraction(1, 1 << 63)


def test_turns_of_given_frequencies(ops):
    freq = [0.0, -1.0, 100.0, 1e-30, 6.283185307179586]
    rc, t = _turns(ops, 2 * len(freq), freq=freq)
    assert rc == 0 and t[0] == 0
    for f, x in zip(freq, t):
        d = (Fraction(x, 1 << 64) - Fraction(f) / TWO_PI) % 1
        assert min(d, 1 - d) <= (abs(Fraction(f)) + 1) * Fraction(1, 1 << 52)
    assert _turns(ops, 2, freq=[math.inf])[0] == -1 and _turns(ops, 2, freq=[math.nan])[0] == -1
    assert _turns(ops, 3)[0] == -1 and _turns(ops, -2)[0] == -1 and _turns(ops, 64, 0.0)[0] == -1 and _turns(ops, 64, math.nan)[0] == -1
    assert ops.lib.mk_rope_turns(0, 1.0, None, None) == 0 and ops.lib.mk_rope_turns(2, 1.0, None, None) == -1


# ------------------------------------------------------------- Python checks
def test_python_checks(ops):
    from speculative_decode_persistent_gb300.mk import MkError
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731

    def bad(fn, status=-1):
        with pytest.raises(MkError) as e:
            fn()
        assert e.value.status == status

    pool5 = (3, 4, 2, 16, 64)
    bad(lambda: ops.KVLayers(h(4, 2, 16, 64), h(4, 2, 16, 64)))
    bad(lambda: ops.KVLayers(h(*pool5), h(2, 4, 2, 16, 64)))
    bad(lambda: ops.KVLayers(h(0, 4, 2, 16, 64), h(0, 4, 2, 16, 64)))
    bad(lambda: ops.KVLayers(h(1, 4, 2, 16, 64).expand(*pool5), h(*pool5)))         # layers over each other
    bad(lambda: ops.KVLayers(h(*pool5), h(6, 4, 2, 16, 64)[::2]))                   # unequally far apart
    bad(lambda: ops.KVLayers(h(*pool5).to(torch.int8), h(*pool5).to(torch.int8)))   # no scales
    sc = h(3, 4, 2, 16, 2)
    bad(lambda: ops.KVLayers(h(*pool5).to(torch.int8), h(*pool5).to(torch.int8), sc, h(6, 4, 2, 16, 2)[::2]))
    bad(lambda: ops.KVLayers(h(*pool5).to(torch.int8), h(*pool5).to(torch.int8), sc[:2], sc[:2]))
    ops.KVLayers(h(6, 4, 2, 16, 64)[::2], h(6, 4, 2, 16, 64)[1::2])
    layers = ops.KVLayers(h(*pool5), h(*pool5))
    bad(lambda: ops.Rope(32, device="cpu"))
    bad(lambda: ops.Rope(-64, device="cpu"))
    bad(lambda: ops.Rope(64, eps=-1.0, device="cpu"))
    bad(lambda: ops.Rope(64, base=0.0, device="cpu"))
    bad(lambda: ops.Rope(64, freq=[1.0], device="cpu"))
    bad(lambda: ops.Rope(64, q_gain=h(64)))
    bad(lambda: ops.Rope(64, q_gain=torch.ones(64), k_gain=torch.ones(128)))
    bad(lambda: ops.Rope(64, q_gain=torch.ones(65)[1:]))
    bad(lambda: ops.Rope(64, q_gain=torch.ones(128)[::2]))
    bad(lambda: ops.Rope(64, q_gain=torch.ones(64, requires_grad=True)))
    rope = ops.Rope(64, device="cpu")
    assert rope.tensors[0].shape == (32,)
    pool, rows = ops.KVPool(h(4, 2, 16, 64), h(4, 2, 16, 64)), ops.KVRows(i(2), i(1), i(1, 3), n_rows=5)
    q, k = h(5, 4, 64), h(5, 2, 64)
    for args in ((q[:4], k, k), (q, k[:4], k), (q, k, h(5, 3, 64)), (q, k, k.float()), (q.double(), k.double(), k.double()),
                 (q[0], k, k), (q.requires_grad_(), k, k), (q.detach(), k, k)):  # the last: not on a CUDA device
        bad(lambda: ops.rope_write(pool, rows, rope, *args))
    lg = torch.zeros(5, 7)
    for args in ((i(5), i(5), lg), (i(5), i(5), lg.double()), (i(5), i(5), lg[:4]), (i(5), i(5), lg[:, ::2]), (i(5), i(5), lg[:, :0]),
                 (i(5), None, lg), (i(4), i(5), lg), (i(5), i(5).long(), lg)):
        bad(lambda: ops.tree_accept(rows, *args))
    bad(lambda: ops.kv_copy(layers, i(3), i(3)))
    bad(lambda: ops.kv_copy(layers, i(3, 1), i(3)))
    bad(lambda: ops.kv_keep(layers, rows, i(5)))
    bad(lambda: ops.kv_keep(layers, rows, i(4)))
    bad(lambda: ops.attend(pool, rows, q.detach(), parents=i(5)))


# ----------------------------------------------------------------- references
def test_references_on_worked_cases():
    from tree_helpers import TreeCase, lineage, turned, walk
    assert lineage([-1, 0, 0, 1, 9, 5]) == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [5]]
    c = TreeCase([(3, 4)], hq=1, hkv=1, dh=64, device="cpu", pad_rows=0, parents=[-1, 0, 0])
    assert c.sees(0, 0, 0).int().tolist() == [[1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 0, 1]]
    assert c.sees(0, 1, 0).int().tolist() == [[0, 1, 0, 0], [0, 0, 1, 0], [0, 0, 0, 1]]
    assert c.sees(0, 1, 1).int().tolist() == [[1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 0, 1]]
    for n in ("k", "v"):
        c.value[n].zero_()
    page = int(c.tables[0, 0])
    for t in range(4):
        c.value["v"][page, 0, t, 0] = 10.0 ** t
    c.q.zero_()
    o, _ = c.tree_ref()
    assert [round(float(x) * n) for x, n in zip(o[:, 0, 0], (2, 3, 3))] == [11, 111, 1011]
    x, _ = turned(torch.tensor([[[3.0, 4.0]]]), [1], 2, torch.tensor([math.pi / 2], dtype=torch.double), None, 0.0)
    assert torch.allclose(x, torch.tensor([[[-4.0, 3.0]]], dtype=torch.double))
    x, _ = turned(torch.tensor([[[3.0, 4.0]]]), [0], 2, torch.zeros(1, dtype=torch.double), torch.tensor([1.0, 2.0]), 0.0)
    assert torch.allclose(x, torch.tensor([[[3.0, 8.0]]], dtype=torch.double) / math.sqrt(12.5))
    lg = [[0.0, 1.0, 1.0], [5.0, 0.0, 0.0], [0.0, 0.0, 2.0]]
    assert walk([-1, 0, 0], [9, 2, 1], lg) == ([0, 2], [1, 2])
    lg[0][0] = math.nan
    assert walk([-1, 0, 0], [9, 2, -1], lg) == ([0], [-1])
