"""rope_write over the whole range of its values: norms where the factor or its product with a gain leaves 32 bits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import assert_within  # noqa: E402
from tree_helpers import TreeCase, turned  # noqa: E402


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def freqs(dims, base=1e7):
    return base ** (-torch.arange(dims // 2, dtype=torch.double, device="cuda") * 2 / max(dims, 1))


def rounded(bound, want, dtype):
    """The bound of a value that is then rounded once to dtype."""
    f = torch.finfo(dtype)
    return bound + (want.abs() + bound) * (f.eps / 2) + f.smallest_normal * f.eps


def single(x):
    """What the call keeps of a number: its nearest in 32 bits."""
    return float(torch.tensor(x, dtype=torch.float32))


SIZES = [1e37, 1e19, 1e15, 1.0, 1e-15, 1e-20, 1e-35, 1e-36, 1e-39, 3e-44]


@pytest.mark.parametrize("gain", [1e-25, 1e-3, 1.0, 1e3, 1e25])
@pytest.mark.parametrize("eps", [1e-6, 2e-30, 9e-31, 1e-34, 1e-38, 1e-44, 0.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_every_size_eps_and_gain(ops, dtype, eps, gain):
    """The factor of a head and its product with a gain may leave 32 bits where the result does not."""
    n = len(SIZES) + 1
    for dh, rot in ((64, 64), (192, 64), (256, 256)):
        c = TreeCase([(n, n)], 2, 1, dh, "f16", dtype, seed=31, pad_rows=0)
        q = torch.randn(n, 2, dh, generator=torch.Generator().manual_seed(dh)).double()
        for i, size in enumerate(SIZES):
            q[i] *= size
        q[n - 1] = torch.sign(q[n - 1]) * torch.finfo(c.dtype).max
        q = q.to(c.dtype).cuda()
        q[:, :, 0] = torch.where((q == 0).all(-1), torch.full_like(q[:, :, 0], torch.finfo(c.dtype).smallest_normal), q[:, :, 0])
        g = (torch.rand(dh, device="cuda") + 0.5) * gain
        pool, rows = c.ops()
        got = ops.rope_write(pool, rows, ops.Rope(rot, 1e4, g, g, eps), q, c.new_k, c.new_v)
        want, b = turned(q, list(range(n)), rot, freqs(rot, 1e4), g, single(eps))
        if dtype == "f32":
            # beside values at 32 bits' end the smallest of a head count as at least 2^-149 of what the largest is scaled
            # to, 1 to 4, before the gain; and values below 2^-126 are multiples of 2^-149, so that each step rounds by up
            # to 2^-150 whatever its size: the two values that are turned (times cosine and sine, 2^1/2 together), one
            # product and one sum, less than 4 of them
            b = b + 2.0 ** -148 * (1 + g.abs().max().double())
        assert_within(got, want, rounded(b, want, c.dtype))
