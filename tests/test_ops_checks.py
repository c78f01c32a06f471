"""The checks of the pool operators' Python calls, each shown by its own message: a call with one fault alone is
refused for that fault. (CPU: what is asked of devices comes last.)"""
import ctypes
import os
import subprocess
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


def h(*s):
    return torch.zeros(s, dtype=torch.float16)


def i(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_layers_contiguous_by_torchs_rule(ops):
    """Strides of dimensions of size 1 say nothing, in a KVLayers as in a KVPool."""
    for views in ([h(3, 4, 16, 1, 64).transpose(2, 3) for _ in "kv"],   # one head
                  [h(3, 2, 1, 16, 64).transpose(1, 2) for _ in "kv"],   # one page
                  [h(2, 16, 1, 1, 128).transpose(1, 3) for _ in "kv"]):  # one of both
        assert all(v[0].is_contiguous() for v in views)
        ops.KVPool(*(v[0] for v in views))
        assert ops.KVLayers(*views).n_layers == views[0].shape[0]
    q = [torch.zeros(3, 4, 16, 1, 64, dtype=torch.int8).transpose(2, 3) for _ in "kv"]
    ops.KVLayers(*q, *(h(3, 4, 16, 1, 2).transpose(2, 3) for _ in "kv"))
    for bad in (h(3, 4, 16, 2, 64).transpose(2, 3), h(3, 2, 4, 16, 64).transpose(1, 2), h(3, 4, 2, 16, 128)[..., ::2], h(3, 4, 2, 64, 16).transpose(3, 4)):
        with pytest.raises(ops.MkError):
            ops.KVLayers(bad, bad.clone(memory_format=torch.preserve_format))


def test_lists_whose_indices_would_leave_32_bits(ops):
    """Kernels step through lists in strides: a list that ends near 2^31 would wrap an index to before its start."""
    from test_tree_ops import _layers, _pool, _rows, _tree
    assert _pool(ops).n_pages
    L = ops.lib
    for n in ((1 << 30) + 1, 2 ** 31 - 1, 2 ** 31 - 65536):
        assert L.mk_kv_copy(_layers(ops), 4096, 4096, n, None) == -8
        assert L.mk_kv_keep(_layers(ops), _rows(ops, n_rows=n), 4096, None, None) == -8
        assert L.mk_tree_accept(_rows(ops, n_rows=n), _tree(ops, work_bytes=1 << 62), None) == -8
        assert L.mk_tree_work_bytes(_rows(ops, n_rows=n), 100) == 0
    assert L.mk_tree_work_bytes(_rows(ops, n_rows=1 << 30), 100) > 0


def test_names_and_tensors(ops):
    """What the module and its handles offered before their marshalling was compiled."""
    assert ops.PAGE_TOKENS == 16 and ops.MK_OPS_MAX_SEQS == 1024
    assert ops.DTYPES == {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    k, v = h(4, 2, 16, 64), h(4, 2, 16, 64)
    pool = ops.KVPool(k, v)
    assert pool.tensors[0] is k and pool.tensors[1] is v and len(pool.tensors) == 2
    assert (pool.device, pool.q8, pool.n_pages, pool.hkv, pool.dh) == (k.device, False, 4, 2, 64)
    q, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), h(4, 2, 16, 2)
    pool = ops.KVPool(q, q, s, s)
    assert len(pool.tensors) == 4 and pool.q8
    assert len(ops.KVLayers(k[None], v[None]).tensors) == 2 and len(ops.KVLayers(q[None], q[None], s[None], s[None]).tensors) == 4
    rows = ops.KVRows(i(3), i(2), i(2, 3), n_rows=5, max_q=4)
    assert (rows.device, rows.n_seqs, rows.n_rows, rows.max_q) == (k.device, 2, 5, 4)


STRUCTS = ("mk_kv_pool", "mk_kv_rows", "mk_dense", "mk_attend_args", "mk_rope", "mk_rope_args", "mk_tree_args", "mk_kv_layers")


def test_ctypes_structures_are_the_headers(ops, tmp_path):
    """The ctypes structures lie in memory as the C compiler lays the header's out."""
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{n} %zu\\n", offsetof({s}, {n}));' for n, _ in getattr(ops, s)._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"mk_ops.h\"\nint main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for s in STRUCTS:
        t = getattr(ops, s)
        assert int(got[s]) == ctypes.sizeof(t), s
        for n, _ in t._fields_:
            assert int(got[f"{s}.{n}"]) == getattr(t, n).offset, (s, n)


def _cases(ops, i, h):
    """(call, what its message says) with one fault each that is found before devices are asked for."""
    pool, rows = ops.KVPool(h(4, 2, 16, 64), h(4, 2, 16, 64)), ops.KVRows(i(2), i(1), i(1, 3), n_rows=5)
    q, k = h(5, 4, 64), h(5, 2, 64)
    rope = ops.Rope(64, device="cpu")
    lg = torch.zeros(5, 7)
    rw = lambda *a, **kw: lambda: ops.rope_write(pool, rows, rope, *a, **kw)  # noqa: E731
    ta = lambda *a: lambda: ops.tree_accept(rows, *a)  # noqa: E731
    at = lambda *a, **kw: lambda: ops.attend(pool, rows, *a, **kw)  # noqa: E731
    return [
        (rw(q[:4], k[:4], k[:4]), "differ from KVRows.n_rows"), (rw(q, k[:4], k), "one number of rows"), (rw(q, k, k[:4]), "one number of rows"),
        (rw(q, k, h(5, 3, 64)), "rope_write v ("), (rw(q, h(5, 2, 128), k), "rope_write k ("), (rw(h(5, 4, 32), k, k), "rope_write q ("),
        (rw(q[0], k, k), "rope_write q ("), (rw(q, k, k.float()), "of one type"), (rw(q.double(), k.double(), k.double()), "float32, float16 or bfloat16"),
        (rw(h(5, 4, 64).requires_grad_(), k, k), "no gradient"), (rw(q, k, k, out=h(1, 4, 64).expand(5, 4, 64)), "must not overlap"),
        (rw(q, k, k, out=h(5, 3, 64)), "rope_write out ("), (rw(h(5, 4, 128)[..., ::2], k, k), "contiguous head dim"), (rw(q, k, None), "(a tensor)"),
        (rw(q, k, k), "one CUDA device"),
        (at(q, out=h(4, 4, 64)), "one number of rows"), (at(q, out=q.float()), "of one type"), (at(q, gate=h(5, 4, 128)), "attend gate ("),
        (at(q, out=h(1, 4, 64).expand(5, 4, 64)), "must not overlap"), (at(q), "one CUDA device"),
        (ta(i(5), i(5), lg.double()), "logits [rows]"), (ta(i(5), i(5), lg[0]), "logits [rows]"), (ta(i(5), i(5), torch.zeros(5, 14)[:, ::2]), "logits [rows]"),
        (ta(i(5), i(5), lg[:, :0]), "logits [rows]"), (ta(i(5), i(5), lg[:4]), "rows of the logits"), (ta(i(5), i(5), lg), "one CUDA device"),
        (ta(i(5), i(5), torch.zeros(9, 5).t()[:, :1]), "one CUDA device"),  # (one logit a row: its stride says nothing)
        (lambda: ops.kv_copy(ops.KVLayers(h(3, 4, 2, 16, 64), h(3, 4, 2, 16, 64)), i(3, 1), i(3)), "kv_copy (int32 [n])"),
        (lambda: ops.kv_copy(ops.KVLayers(h(3, 4, 2, 16, 64), h(3, 4, 2, 16, 64)), i(3), i(3)), "a CUDA device"),
        (lambda: ops.kv_keep(ops.KVLayers(h(3, 4, 2, 16, 64), h(3, 4, 2, 16, 64)), rows, i(5)), "one CUDA device"),
        (lambda: ops.kv_keep(pool, rows, i(5)), "handle"), (lambda: ops.attend(rows, pool, q), "handle"), (lambda: ops.attend(pool, rows, [1]), "(a tensor)"),
    ]


def test_each_fault_by_its_own_message(ops):
    for n, (call, says) in enumerate(_cases(ops, i, h)):
        with pytest.raises(ops.MkError) as e:
            call()
        assert e.value.status == -1 and says in str(e.value), (n, says, str(e.value))
