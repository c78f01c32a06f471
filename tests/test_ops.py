"""KV-cache operators on the CPU: exports, the C entries' refusals (all made
before any device work) and the Python checks."""
import ctypes
import os
import re
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "tests"))


@pytest.fixture(scope="module")
def ops():
    from speculative_decode_persistent_gb300 import build as b
    b.build()
    from speculative_decode_persistent_gb300 import ops as o
    return o


def test_exports_every_declared_symbol(ops):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mk_ops.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mk_[a-z_]+)\s*\(", src)))
    assert names == sorted(ops.EXPORTS)
    for n in names:
        assert hasattr(ops.lib, n)


def _pool(ops, **kw):
    p = ops.mk_kv_pool(4096, 8192, 0, 0, 0, 8, 2, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _rows(ops, **kw):
    r = ops.mk_kv_rows(4096, 4096, 4096, 1, 4, 2, 4)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


BAD_POOL = [(dict(k=None), -1), (dict(v=0), -1), (dict(k=4100), -1), (dict(n_pages=0), -1), (dict(hkv=0), -1),
            (dict(kv_dtype=2), -1), (dict(kv_dtype=1), -1), (dict(kv_dtype=1, k_scale=4096, v_scale=4098), -1),
            (dict(dh=0), -1), (dict(dh=32), -8), (dict(dh=320), -8), (dict(n_pages=1 << 27), -8)]
BAD_ROWS = [(dict(row_start=None), -1), (dict(kv_len=None), -1), (dict(tables=None), -1), (dict(n_seqs=-1), -1),
            (dict(n_rows=-1), -1), (dict(table_stride=-1), -1), (dict(n_seqs=1025), -8), (dict(table_stride=1 << 28), -8)]


@pytest.mark.parametrize("pool_kw,rows_kw,status", [(p, {}, s) for p, s in BAD_POOL] + [({}, r, s) for r, s in BAD_ROWS])
def test_entries_refuse_bad_pools_and_rows(ops, pool_kw, rows_kw, status):
    p, r = _pool(ops, **pool_kw), _rows(ops, **rows_kw)
    d = ops.mk_dense(4096, 128, 64)
    assert ops.lib.mk_kv_write(p, r, d, d, 1, None) == status
    assert ops.lib.mk_kv_read(p, r, d, d, 1, None) == status
    assert ops.lib.mk_attend_work_bytes(p, r, 4) == 0
    a = _args(ops)
    assert ops.lib.mk_attend(p, r, a, None) == status


def _args(ops, **kw):
    d = ops.mk_dense(4096, 256, 64)
    a = ops.mk_attend_args(d, ops.mk_dense(), d, 4, 1, 0.125, 0, 0, 4096, 1 << 40)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), -1), (dict(hq=3), -1), (dict(hq=514), -8), (dict(dtype=0), -1), (dict(dtype=3), -1), (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(window=-1), -1),
    (dict(sinks=-1, window=4), -1), (dict(sinks=4), -1), (dict(work=None), -1), (dict(work=4100), -1),
    (dict(work_bytes=0), -1)])
def test_attend_refuses_bad_arguments(ops, kw, status):
    assert ops.lib.mk_attend(_pool(ops), _rows(ops), _args(ops, **kw), None) == status


def test_attend_refuses_bad_tensors(ops):
    for name in ("q", "out", "gate"):
        a = _args(ops)
        setattr(a, name, ops.mk_dense(4097, 256, 64))
        assert ops.lib.mk_attend(_pool(ops), _rows(ops), a, None) == -1
    for name in ("q", "out"):
        a = _args(ops)
        setattr(a, name, ops.mk_dense(None, 256, 64))
        assert ops.lib.mk_attend(_pool(ops), _rows(ops), a, None) == -1
    assert ops.lib.mk_attend(_pool(ops), _rows(ops), None, None) == -1


def test_write_and_read_refuse_bad_tensors(ops):
    d, odd = ops.mk_dense(4096, 128, 64), ops.mk_dense(4097, 128, 64)
    for fn in (ops.lib.mk_kv_write, ops.lib.mk_kv_read):
        assert fn(_pool(ops), _rows(ops), d, odd, 1, None) == -1
        assert fn(_pool(ops), _rows(ops), d, ops.mk_dense(None, 128, 64), 1, None) == -1
        assert fn(_pool(ops), _rows(ops), None, d, 1, None) == -1
        assert fn(_pool(ops), _rows(ops), d, d, 3, None) == -1


def test_nothing_to_do_is_ok_without_a_device(ops):
    d = ops.mk_dense(None, 128, 64)
    for kw in (dict(n_seqs=0), dict(n_rows=0)):
        assert ops.lib.mk_kv_write(_pool(ops), _rows(ops, **kw), d, d, 1, None) == 0
        assert ops.lib.mk_kv_read(_pool(ops), _rows(ops, **kw), d, d, 1, None) == 0
        a = _args(ops, q=d, out=d)
        assert ops.lib.mk_attend(_pool(ops), _rows(ops, **kw), a, None) == 0


def test_python_checks(ops):
    from speculative_decode_persistent_gb300.mk import MkError
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731

    def bad(fn):
        with pytest.raises(MkError) as e:
            fn()
        assert e.value.status == -1

    bad(lambda: ops.KVPool(h(4, 2, 8, 64), h(4, 2, 8, 64)))
    bad(lambda: ops.KVPool(h(4, 2, 16, 64), h(3, 2, 16, 64)))
    bad(lambda: ops.KVPool(h(4, 2, 16, 64).float(), h(4, 2, 16, 64).float()))
    bad(lambda: ops.KVPool(h(4, 2, 16, 64), h(4, 2, 16, 64), h(4, 2, 16, 2), h(4, 2, 16, 2)))
    bad(lambda: ops.KVPool(h(4, 2, 16, 64).to(torch.int8), h(4, 2, 16, 64).to(torch.int8)))
    bad(lambda: ops.KVPool(h(4, 2, 16, 64).to(torch.int8), h(4, 2, 16, 64).to(torch.int8), h(4, 2, 16, 1), h(4, 2, 16, 1)))
    bad(lambda: ops.KVPool(h(4, 16, 2, 64).transpose(1, 2), h(4, 16, 2, 64).transpose(1, 2)))
    bad(lambda: ops.KVRows(i(2), i(2), i(2, 3)))
    bad(lambda: ops.KVRows(i(3).long(), i(2), i(2, 3)))
    bad(lambda: ops.KVRows(i(3), i(2), i(1, 3)))
    bad(lambda: ops.KVRows(i(3), i(2), i(2, 6)[:, ::2]))
    bad(lambda: ops.KVRows(i(3), i(2), i(2, 3), n_rows=-1))
    pool, rows = ops.KVPool(h(4, 2, 16, 64), h(4, 2, 16, 64)), ops.KVRows(i(2), i(1), i(1, 3), n_rows=5)
    bad(lambda: ops.attend(pool, rows, h(5, 4, 32)))               # head dim
    bad(lambda: ops.attend(pool, rows, h(5, 256)))                 # rank
    bad(lambda: ops.attend(pool, rows, h(4, 4, 64)))               # rows
    bad(lambda: ops.attend(pool, rows, h(5, 4, 128)[..., ::2]))    # head dim not contiguous
    bad(lambda: ops.attend(pool, rows, h(5, 4, 64), gate=h(5, 2, 64)))
    bad(lambda: ops.attend(pool, rows, h(5, 4, 64), gate=h(5, 4, 64).bfloat16()))
    bad(lambda: ops.attend(pool, rows, h(5, 4, 64), out=h(1, 4, 64).expand(5, 4, 64)))
    bad(lambda: ops.attend(pool, rows, h(5, 4, 64).requires_grad_()))
    bad(lambda: ops.attend(pool, rows, h(5, 4, 64)))               # not on a CUDA device
    bad(lambda: ops.kv_write(pool, rows, h(5, 2, 64), h(5, 2, 64).float()))
    bad(lambda: ops.kv_write(pool, rows, h(5, 3, 64), h(5, 3, 64)))
    bad(lambda: ops.kv_write(pool, rows, h(5, 2, 64).double(), h(5, 2, 64).double()))
    bad(lambda: ops.kv_read(pool, ops.KVRows(i(2), i(1), i(1, 3))))
    bad(lambda: ops.kv_read(pool, rows, out=(h(5, 2, 64), h(1, 2, 64).expand(5, 2, 64))))


def test_reference_against_a_worked_case():
    """The 64-bit reference itself: two tokens, one head, values by hand."""
    import math
    from ops_helpers import Case
    c = Case([(2, 2)], hq=1, hkv=1, dh=64, device="cpu", pad_rows=0)
    page = int(c.tables[0, 0])
    for n in ("k", "v"):
        c.value[n].zero_()
    c.value["k"][page, 0, 1, 0] = 8.0
    c.value["v"][page, 0, 0, 0], c.value["v"][page, 0, 1, 0] = 1.0, 3.0
    c.q.zero_()
    c.q[1, 0, 0] = 1.0
    o, _ = c.attend_ref()
    w = math.e / (1 + math.e)  # score 8 / sqrt(64) = 1 against 0
    assert float(o[0, 0, 0]) == 1.0
    assert abs(float(o[1, 0, 0]) - (1 * (1 - w) + 3 * w)) < 1e-12
    o, _ = c.attend_ref(window=1)
    assert float(o[1, 0, 0]) == 3.0
    o, _ = c.attend_ref(window=1, sinks=1)
    assert abs(float(o[1, 0, 0]) - (1 * (1 - w) + 3 * w)) < 1e-12
