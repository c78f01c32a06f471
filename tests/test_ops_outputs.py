"""Which strides an output of the KV-cache operators may have (CPU): every layout whose rows do not
overlap, [heads][rows][head dim] among them. The operators refuse CPU tensors after this check, so the
error's text tells how far a call got."""
import itertools

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from speculative_decode_persistent_gb300 import build as b
    b.build()
    from speculative_decode_persistent_gb300 import ops as o
    return o


def _text(ops, n, heads, dh, out):
    from speculative_decode_persistent_gb300.mk import MkError
    pool = ops.KVPool(*(torch.zeros((4, 1, 16, dh), dtype=torch.float16) for _ in "kv"))
    rows = ops.KVRows(*(torch.zeros(s, dtype=torch.int32) for s in ((2,), (1,), (1, 3))), n_rows=n)
    with pytest.raises(MkError) as e:
        ops.attend(pool, rows, torch.zeros((n, heads, dh), dtype=torch.float16), out=out)
    return str(e.value)


def test_heads_first_outputs_are_taken(ops):
    out = torch.empty((2, 5, 64), dtype=torch.float16).transpose(0, 1)
    assert "one CUDA device" in _text(ops, 5, 2, 64, out)
    pool = ops.KVPool(*(torch.zeros((4, 2, 16, 64), dtype=torch.float16) for _ in "kv"))
    rows = ops.KVRows(*(torch.zeros(s, dtype=torch.int32) for s in ((2,), (1,), (1, 3))), n_rows=5)
    with pytest.raises(Exception, match="one CUDA device"):
        ops.kv_read(pool, rows, out=(out, out.clone()))


@pytest.mark.parametrize("n,heads", [(1, 1), (1, 4), (4, 1), (2, 2), (3, 2), (2, 3), (5, 4)])
def test_outputs_are_refused_exactly_when_they_overlap(ops, n, heads):
    dh = 64
    flat = torch.empty(1 << 14, dtype=torch.float16)
    steps = (0, 1, 32, 63, 64, 65, 96, 128, 130, 192, 256, 320, 384, 640)
    for row, head in itertools.product(steps, steps):
        at = sorted(r * row + h * head for r in range(n) for h in range(heads))
        overlap = any(b - a < dh for a, b in zip(at, at[1:]))
        text = _text(ops, n, heads, dh, flat.as_strided((n, heads, dh), (row, head, 1)))
        assert ("overlap" in text) == overlap, (row, head, text)
