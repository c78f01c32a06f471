"""The checks of the pool operators' Python calls, each shown by its own message: a call with one fault alone is
refused for that fault. (CPU: what is asked of devices comes last.)"""
import os
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
