"""rope_write of many rows in every type, head dim and layout, and the rotation of the fused step beside it."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import NP, assert_within, half_even  # noqa: E402
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


VARIANTS = [(64, 64, 9, 1), (64, 64, 30, 2), (128, 64, 5, 2), (128, 128, 14, 2), (192, 192, 3, 2), (192, 128, 6, 2), (256, 64, 4, 3), (256, 256, 24, 4)]


def rows_for(dh, heads, batches):
    """As many rows as need `batches` times a group's four (two of fp32) in each of the blocks that are resident at once."""
    groups = 256 // (4 if dh == 64 else 8 if dh == 128 else 16)
    blocks = -(-heads // groups)
    per = groups // -(-heads // blocks)
    return max(400 * groups // heads + 1, -(-304 * batches // blocks) * per * 4 - 3)


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dh,rot,hq,hkv", VARIANTS)
def test_many_rows(ops, dh, rot, hq, hkv, dtype, kv, odd):
    """More rows than one a group, over several batches a block; heads whose squares leave 32 bits all over them."""
    heads = hq + 2 * hkv
    n = min(rows_for(dh, heads, 1 if odd else 12 if hq == 30 else 3), 60000000 // (heads * dh))
    seqs = [(n // 3, n // 3 + 40), (0, 3), (n - n // 3, n - n // 3)]
    t, g = NP[dtype], torch.Generator(device="cuda").manual_seed(n)
    c = TreeCase(seqs, 1, hkv, dh, kv, "f16", seed=dh + hq, pad_rows=3, kind="star")
    before = {x: p.clone() for x, p in c.pool.items()}
    shift = 1 if odd else 0
    flat = torch.randn(c.n_rows * heads * dh + shift, generator=g, device="cuda")
    qkv = flat[shift:].view(c.n_rows, heads, dh)
    if dtype != "f16":
        pick = torch.rand(c.n_rows, hq + hkv, 1, generator=g, device="cuda")
        qkv[:, :hq + hkv] *= torch.where(pick < 0.03, 1e20, torch.where(pick > 0.98, 1e-25, 1.0))
    flat = flat.to(t)
    qkv = flat[shift:].view(c.n_rows, heads, dh)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    gq, gk = torch.rand(dh, device="cuda") + 0.5, torch.rand(dh, device="cuda") + 0.5
    eps = 1e-38
    pool, rows = c.ops()
    was = q.clone()
    flat_out = torch.full((c.n_rows * hq * dh + shift,), 7.0, device="cuda", dtype=t)
    out = ops.rope_write(pool, rows, ops.Rope(rot, 1e4, gq, gk, eps), q, k, v, out=flat_out[shift:].view(c.n_rows, hq, dh))
    u, pos = c.rows_used, [p for m, T in seqs for p in range(T - m, T)]
    assert torch.equal(q, was) and bool((out[u:] == 7).all())
    want, b = turned(q[:u], pos, rot, freqs(rot, 1e4), gq, single(eps))
    assert_within(out[:u], want, rounded(b, want, t))
    del want, b
    seq = torch.tensor([i for i, (m, _) in enumerate(seqs) for _ in range(m)], device="cuda")
    slot = torch.tensor(pos, device="cuda")
    page = c.tables.long()[seq, slot // 16]
    at = lambda x: x[page, :, slot % 16].double()  # noqa: E731
    wk, bk = turned(k[:u], pos, rot, freqs(rot, 1e4), gk, single(eps))
    for name, x, bd in (("k", wk, bk), ("v", v[:u].double(), torch.zeros_like(bk))):
        if kv == "f16":
            assert_within(at(c.pool[name]), x, rounded(bd, x, torch.float16))
            continue
        d, code = at(c.pool[name + "_scale"]), at(c.pool[name])
        ax, ab = x.unflatten(-1, (-1, 32)).abs().amax(-1) / 127, bd.unflatten(-1, (-1, 32)).amax(-1) / 127
        assert bool((d >= half_even((ax - ab).clamp_min(0))).all()) and bool((d <= half_even(ax + ab)).all())
        d32 = d.repeat_interleave(32, -1)
        # the nearest code, clamped at 127 where the scale was rounded down (by at most half a step of binary16)
        err = (code * d32 - x).abs()
        assert bool((err <= d32 / 2 * (1 + 1e-12) + 127 * (d32 * 2.0 ** -11 + 2.0 ** -25) + bd).all())
        assert bool((err <= d32 / 2 * (1 + 1e-12) + bd)[(code.abs() < 127) & (d32 > 0)].all())
    used = torch.zeros(c.n_pages, 16, dtype=torch.bool, device="cuda")
    used[page, slot % 16] = True
    for name, x in before.items():
        a, w = c.pool[name].transpose(1, 2)[~used], x.transpose(1, 2)[~used]
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(w)), name


def test_the_fused_steps_rotation(ops):
    """A row that the fused step caches at a position is the one that it caches at position 0, turned there by
    rope_write: both may write one pool."""
    from gen import configs
    from gen.synth import make_weights
    from speculative_decode_persistent_gb300 import mk
    model = dict(configs.TINY, kinds=[1, 0, 0, 0])  # attention first: K of the first layer is the token's own
    eng = mk.Engine(model, make_weights(model, 0), 0, 1300)
    hkv, dh = model["hkv"], model["dh"]
    rope = ops.Rope(dh, model["rope_base"], device="cuda")

    def cached(p, token):
        if p:
            z = torch.zeros(1, p, hkv, dh, device="cuda", dtype=torch.float16)
            eng.seq_load(0, z, z)
        else:
            eng.seq_new(0)
        eng.step([token], [p], [0])
        eng.commit([0], [1])
        return eng.seq_kv(0, torch.float32)[0][:, p]

    for token in (7, 1234):
        k0 = cached(0, token)
        assert float(k0.abs().max()) > 0
        for p in (1, 2, 63, 1000, 20001):
            want = cached(p, token)
            pool = ops.KVPool(*(torch.zeros(1, hkv, 16, dh, device="cuda", dtype=torch.float16) for _ in "kv"))
            i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
            rows = ops.KVRows(i(0, 1), i(1), i(0)[None], n_rows=1)
            ops.rope_write(pool, rows, rope, k0, k0, k0, positions=i(p))
            got = ops.kv_read(pool, rows, torch.float32)[0]
            # k0 was rounded to binary16 (half a step, 2^-11, of each of a turned pair), and so is each of the two results
            pair = k0.abs() + torch.cat([k0[..., dh // 2:], k0[..., :dh // 2]], -1).abs()
            assert bool(((got - want).abs() <= 2.0 ** -11 * (pair + got.abs() + want.abs()) * 1.001 + 2.0 ** -24).all()), (token, p)
    eng.close()
