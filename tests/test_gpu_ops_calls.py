"""Calls of the KV-cache operators around the GPU work: outputs in other layouts."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import Case, assert_within  # noqa: E402,F401


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_outputs_with_heads_first(ops, kv):
    """[heads][rows][head dim] seen as [rows][heads][head dim], with gaps and without."""
    c = Case([(9, 300), (140, 141)], 6, 2, 128, kv, "f16", seed=50, pad_rows=0)
    pool, rows = c.ops()
    want = ops.attend(pool, rows, c.q, gate=c.gate)
    k, v = ops.kv_read(pool, rows)
    for gap in (0, 3):
        make = lambda h: torch.full((h, c.n_rows + gap, 128), 7.0, dtype=c.dtype, device="cuda")  # noqa: E731
        o, ok, ov = make(6), make(2), make(2)
        view = lambda t: t[:, :c.n_rows].transpose(0, 1)  # noqa: E731
        ops.attend(pool, rows, c.q, gate=c.gate, out=view(o))
        ops.kv_read(pool, rows, out=(view(ok), view(ov)))
        assert torch.equal(view(o), want) and torch.equal(view(ok), k) and torch.equal(view(ov), v)
        for t in (o, ok, ov):
            assert bool((t[:, c.n_rows:] == 7).all())
