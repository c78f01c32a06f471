"""KV-cache operators on the GPU against a 64-bit reference (tests/ops_helpers.py):
every pool and dense type, head layouts, lengths from one token on, windows
and sinks, rows that see nothing, NaN and infinities in unseen places, odd
strides and alignments, rows behind the last sequence, missing pages, graph
capture, other streams, pools beyond 32-bit offsets, and the operators
together on an engine's pool."""
import math
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ops_helpers import Case, assert_within, q8_values  # noqa: E402


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.float16 else t


# ------------------------------------------------------------------- write
WRITES = [([(1, 1)], 1, 64), ([(1, 17), (3, 3), (16, 32)], 2, 128), ([(7, 40), (0, 5), (33, 33)], 3, 192),
          ([(130, 1000), (1, 16)], 4, 256)]


def _check_written(c, before, codes_exact=True):
    """The pool holds the new rows where their positions lie, and nothing else changed."""
    touched = torch.zeros(c.n_pages, 16, dtype=torch.bool, device="cuda")
    for i, (n, T) in enumerate(c.seqs):
        for j in range(n):
            p = T - n + j
            page = int(c.tables[i, p // 16]) if p >= 0 else -1
            if not 0 <= page < c.n_pages:
                continue
            touched[page, p % 16] = True
            r = int(c.start[i]) + j
            for name, x in (("k", c.new_k[r]), ("v", c.new_v[r])):
                got = c.pool[name][page, :, p % 16]
                if c.kv == "f16":
                    assert torch.equal(bits(got), bits(x.half())), (i, j, name)
                else:
                    codes, d = q8_values(x)
                    assert torch.equal(got, codes.to(torch.int8)), (i, j, name)
                    assert torch.equal(bits(c.pool[name + "_scale"][page, :, p % 16]), bits(d.half())), (i, j, name)
    for name, was in before.items():
        now = c.pool[name].transpose(1, 2)
        assert torch.equal(bits(now)[~touched], bits(was.transpose(1, 2))[~touched]), name


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("seqs,hkv,dh", WRITES)
def test_write(ops, seqs, hkv, dh, dtype, kv):
    c = Case(seqs, hq=hkv, hkv=hkv, dh=dh, kv=kv, dtype=dtype, seed=1)
    before = {n: t.clone() for n, t in c.pool.items()}
    pool, rows = c.ops()
    ops.kv_write(pool, rows, c.new_k, c.new_v)
    _check_written(c, before)


@pytest.mark.parametrize("amp", [1e-7, 1e-4, 30.0, 1e4])
def test_write_q8_scales_of_every_size(ops, amp):
    """Subnormal scales, ties of the scale and of the codes (values on a grid), zero blocks."""
    c = Case([(64, 64)], hkv=2, dh=64, kv="q8", dtype="f32", seed=2)
    c.new_k.mul_(amp)
    c.new_v.copy_(torch.round(c.new_v * 8) / 2 * amp)
    c.new_v[3] = 0
    c.new_v[5, 0, :32] = (torch.arange(32, device="cuda") - 15.5) * amp
    c.new_v[5, 0, 31] = 127 * amp
    before = {n: t.clone() for n, t in c.pool.items()}
    ops.kv_write(*c.ops(), c.new_k, c.new_v)
    _check_written(c, before)


def test_write_equals_the_step_codec(ops):
    from speculative_decode_persistent_gb300 import mk
    from test_gpu_q8_codec import _blocks
    x = torch.from_numpy(_blocks()).cuda()
    n = x.shape[0] // 2 * 2
    c = Case([(n // 2, n // 2)], hkv=1, dh=64, kv="q8", dtype="f32", pad_rows=0)
    c.new_k.copy_(x[:n].view(n // 2, 1, 64))
    ops.kv_write(*c.ops(), c.new_k, c.new_k)
    q, d = mk.q8_encode(x[:n])
    page = c.tables[0].long().repeat_interleave(16)[:n // 2]
    slot = torch.arange(n // 2, device="cuda") % 16
    assert torch.equal(c.pool["k"][page, 0, slot].reshape(n, 32), q)
    assert torch.equal(bits(c.pool["k_scale"][page, 0, slot]).reshape(n), d)


def test_write_drops_rows_without_a_page_or_position(ops):
    c = Case([(20, 20), (6, 20)], kv="q8", dtype="f32")
    c.tables[0, 0], c.tables[1, 1] = -1, c.n_pages  # no page; out of range
    before = {n: t.clone() for n, t in c.pool.items()}
    ops.kv_write(*c.ops(), c.new_k, c.new_v)
    _check_written(c, before)
    c = Case([(5, 5)], kv="f16", dtype="f32")
    c.kv_len[0] = 2  # more rows than tokens: three of them have no position
    c.seqs = [(5, 2)]
    before = {n: t.clone() for n, t in c.pool.items()}
    ops.kv_write(*c.ops(), c.new_k, c.new_v)
    _check_written(c, before)


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("seqs,hkv,dh", WRITES)
def test_read(ops, seqs, hkv, dh, dtype, kv):
    c = Case(seqs, hq=hkv, hkv=hkv, dh=dh, kv=kv, dtype=dtype, seed=3)
    pool, rows = c.ops()
    out = tuple(torch.full((c.n_rows, hkv, dh), 7.0, dtype=c.dtype, device="cuda") for _ in "kv")
    ops.kv_read(pool, rows, out=out)
    for name, got in zip("kv", out):
        at = 0
        for i, (n, T) in enumerate(seqs):
            want = c.gather(i, name)[0][T - n:]
            # a binary16 or code x scale value fits fp32 exactly: one rounding
            assert torch.equal(got[at:at + n], want.float().to(c.dtype))
            at += n
        assert bool((got[at:] == 7.0).all())  # rows behind the last sequence


def test_read_holes_and_negative_positions(ops):
    c = Case([(20, 20), (6, 20)], kv="f16", dtype="f32")
    c.tables[0, 1] = -5
    c.kv_len[1] = 4
    k, v = ops.kv_read(*c.ops(), torch.float32)
    assert not k[16:22].any() and not v[16:22].any()
    page = int(c.tables[1, 0])
    assert torch.equal(k[22:26], c.pool["k"][page, :, :4].transpose(0, 1).float())


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_strided_and_unaligned_dense_tensors(ops, kv):
    c = Case([(9, 30), (4, 4)], hkv=2, dh=128, kv=kv, dtype="bf16", pad_rows=0)
    pool, rows = c.ops()
    ops.kv_write(pool, rows, c.new_k, c.new_v)
    want = {n: t.clone() for n, t in c.pool.items()}
    # the same values in other layouts: [heads][rows][dh], an odd element offset, rows with gaps
    hk = c.new_k.transpose(0, 1).contiguous().transpose(0, 1)
    flat = torch.empty(c.new_v.numel() + 1, dtype=c.dtype, device="cuda")[1:]
    hv = flat.view_as(c.new_v).copy_(c.new_v)
    for k, v in ((hk, hv), (hv * 0 + c.new_k, hv), (torch.nn.functional.pad(c.new_k, (0, 5))[..., :128], c.new_v)):
        for n in ("k", "v"):
            c.pool[n].zero_()
        before = {n: t.clone() for n, t in c.pool.items()}
        ops.kv_write(pool, rows, k, v)
        _check_written(c, before)
    ref = ops.kv_read(pool, rows, torch.bfloat16)
    gap = torch.full((c.n_rows, 2, 133), 3.0, dtype=torch.bfloat16, device="cuda")
    odd = torch.empty(c.n_rows * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(c.n_rows, 2, 128)
    ops.kv_read(pool, rows, out=(gap[..., :128], odd))
    assert torch.equal(gap[..., :128], ref[0]) and torch.equal(odd, ref[1]) and bool((gap[..., 128:] == 3).all())
    # one row for all: a broadcast input
    one = c.new_k[:1].expand(c.n_rows, 2, 128)
    ops.kv_write(pool, rows, one, one)
    k, v = ops.kv_read(pool, rows, torch.float32)
    assert torch.equal(k, k[:1].expand_as(k)) and torch.equal(k, v)
    assert want["k"].shape == c.pool["k"].shape


# ------------------------------------------------------------------ attend
def check_attend(ops, c, window=0, sinks=0, gate=False, **kw):
    pool, rows = c.ops()
    out = torch.full_like(c.q, 5.0)
    ops.attend(pool, rows, c.q, window=window, sinks=sinks, gate=c.gate if gate else None, out=out, **kw)
    want, bound = c.attend_ref(window, sinks, gate, scale=kw.get("scale"))
    assert_within(out[:c.rows_used], want, bound)
    assert bool((out[c.rows_used:] == 5.0).all())  # rows behind the last sequence
    return out


SHAPES = [
    # seqs, hq, hkv, dh
    ([(1, 1)], 1, 1, 64), ([(1, 15), (1, 16), (1, 17)], 4, 2, 64), ([(1, 127), (1, 128), (1, 129), (1, 400)], 6, 1, 128),
    ([(3, 700), (1, 1), (8, 8), (5, 260)], 6, 2, 192), ([(1, 4097)], 24, 4, 256), ([(3, 1000), (3, 77)], 24, 4, 256),
    ([(8, 300)], 32, 1, 64), ([(130, 130)], 1, 1, 128), ([(64, 515), (2, 2), (100, 100)], 12, 2, 256),
    ([(257, 600), (1, 3)], 8, 8, 128), ([(200, 333)], 5, 1, 192), ([(300, 2000), (0, 9), (43, 43)], 12, 2, 256),
    ([(90, 90)], 48, 1, 64), ([(2, 200)], 130, 1, 128), ([(1, 60)], 256, 1, 256)]


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("seqs,hq,hkv,dh", SHAPES)
def test_attend_causal(ops, seqs, hq, hkv, dh, dtype, kv):
    check_attend(ops, Case(seqs, hq, hkv, dh, kv, dtype, seed=4))


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (127, 4), (128, 16), (129, 130), (300, 1), (500, 700), (10**9, 3)])
@pytest.mark.parametrize("seqs,hq,hkv,dh", [([(1, 900), (5, 1300), (1, 1)], 6, 2, 64), ([(150, 1000), (70, 70)], 12, 2, 256),
                                            ([(200, 640)], 2, 2, 128)])
def test_attend_window_and_sinks(ops, seqs, hq, hkv, dh, window, sinks, kv):
    check_attend(ops, Case(seqs, hq, hkv, dh, kv, "f16", seed=5), window, sinks, gate=sinks == 4)


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("dh,hq,hkv", [(64, 4, 2), (128, 8, 2), (192, 3, 1), (256, 6, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_attend_missing_pages_and_empty_rows(ops, dh, hq, hkv, kv, window, sinks):
    """Released pages (-1, out of range) are unseen; rows that see nothing give 0; so do rows
    at negative positions and sequences of no token."""
    c = Case([(70, 400), (20, 20), (4, 300), (3, 3)], hq, hkv, dh, kv, "f16", seed=6)
    c.tables[0, 2], c.tables[0, 7:20], c.tables[0, 24] = -1, -1, c.n_pages + 7
    c.tables[1, :] = -1          # nothing left: every row is empty
    c.tables[2, 18] = -3         # the rows' own page is gone
    out = check_attend(ops, c, window, sinks)
    assert not out[70:90].any()
    c = Case([(5, 5), (2, 2)], hq, hkv, dh, kv, "f16", seed=7)
    c.kv_len[0], c.kv_len[1] = 2, 0
    pool, rows = c.ops()
    out = ops.attend(pool, rows, c.q, window=window, sinks=sinks)
    assert not out[:3].any() and not out[5:7].any() and bool(torch.isfinite(out[:7]).all())
    c.seqs, c.rows_used = [(2, 2)], 2
    c.q = c.q[3:]
    want, bound = c.attend_ref(window, sinks)
    assert_within(out[3:5], want, bound)


@pytest.mark.parametrize("dh,hq,hkv,n", [(64, 4, 2, 40), (128, 4, 1, 90), (256, 6, 1, 60), (192, 2, 1, 150)])
@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_nan_and_inf_in_unseen_places(ops, dh, hq, hkv, n, kv, window):
    """A NaN or infinite K or V of a token reaches the rows that see it, in its own dim, and no other row."""
    c = Case([(n, n + 60), (3, 50)], hq, hkv, dh, kv, "f16", seed=8)
    first = 60

    def put(name, pos, head, dim, x):
        page = int(c.tables[0, pos // 16])
        if kv == "f16":
            c.pool[name][page, head, pos % 16, dim] = x
            c.value[name][page, head, pos % 16, dim] = x
        else:  # an infinite or NaN scale takes its whole block
            b = dim // 32
            c.pool[name][page, head, pos % 16, 32 * b:32 * b + 32] = 1
            c.pool[name + "_scale"][page, head, pos % 16, b] = x
            c.value[name][page, head, pos % 16, 32 * b:32 * b + 32] = x

    put("v", first + n - 2, 0, 3, math.inf)      # seen by the last two rows only
    put("v", first + n // 2, 0, 40, math.nan)    # by the later half
    put("v", first + n - 9, 0, 3, -math.inf)
    put("v", 5, 0, 9, math.inf)                  # an old token: by all, or outside the window of the later rows
    put("k", first + n - 4, hkv - 1, 0, math.nan)
    check_attend(ops, c, window)


def test_attend_infinite_scores(ops):
    """-inf scores weigh nothing; a row that has only them gives 0; +inf or NaN queries give NaN."""
    c = Case([(6, 40)], 2, 1, 64, "f16", "f16", seed=9)
    for i in range(40):
        page = int(c.tables[0, i // 16])
        for n in (c.pool, c.value):
            n["k"][page, 0, i % 16, 0] = -math.inf if i < 38 else 1.0
    c.q[:, :, 0] = 1.0
    c.q[5, 1, 7] = math.nan
    out = check_attend(ops, c)
    assert not out[:4].any() and bool(out[4].any()) and bool(torch.isnan(out[5, 1]).all())


@pytest.mark.parametrize("amp", [1e-30, 1e-6, 1.0, 3e4, 1e20])
def test_attend_bf16_queries_of_every_size(ops, amp):
    """bf16 reaches far beyond binary16: the operands are scaled by powers of two. The score scale undoes amp."""
    c = Case([(9, 200)], 4, 2, 128, "f16", "bf16", seed=10)
    c.q.mul_(amp)
    c.q[2, 1] = 0
    check_attend(ops, c, scale=1.0 / (amp * math.sqrt(128)) if amp > 1e-20 else 1.0)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_attend_scales(ops, scale):
    """Nearly uniform to nearly one-hot probabilities: the running maximum moves a lot."""
    check_attend(ops, Case([(40, 700), (2, 300)], 6, 1, 128, "f16", "f16", seed=11), scale=scale)


def test_attend_growing_scores(ops):
    """Every block of tokens holds larger scores than the last: each one moves the maximum."""
    for dh, hq, q in ((64, 2, 3), (256, 6, 100)):
        c = Case([(q, 1500)], hq, 1, dh, "f16", "f16", seed=12)
        ramp = torch.arange(1500, device="cuda") / 150.0
        page = c.tables[0].long().repeat_interleave(16)[:1500]
        slot = torch.arange(1500, device="cuda") % 16
        for n in (c.pool, c.value):
            n["k"][page, 0, slot, 0] = (ramp * dh ** 0.5).to(n["k"].dtype)
        c.value["k"] = c.pool["k"].double()
        c.q[..., 0] = 4.0
        check_attend(ops, c)


def test_attend_strides_alignment_and_in_place(ops):
    c = Case([(9, 300), (40, 41)], 6, 2, 128, "f16", "bf16", seed=13, pad_rows=0)
    pool, rows = c.ops()
    want = ops.attend(pool, rows, c.q, gate=c.gate)
    n = c.n_rows
    heads_first = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.empty(c.q.numel() + 1, dtype=c.dtype, device="cuda")[1:].view_as(c.q).copy_(c.q)
    gap = torch.nn.functional.pad(c.q, (0, 3))[..., :128]
    for q in (heads_first, odd, gap):
        assert torch.equal(ops.attend(pool, rows, q, gate=c.gate), want)
    for g in (c.gate.transpose(0, 1).contiguous().transpose(0, 1),
              torch.empty(c.q.numel() + 1, dtype=c.dtype, device="cuda")[1:].view_as(c.q).copy_(c.gate)):
        assert torch.equal(ops.attend(pool, rows, c.q, gate=g), want)
    out = torch.full((n, 6, 133), 2.0, dtype=c.dtype, device="cuda")
    ops.attend(pool, rows, c.q, gate=c.gate, out=out[..., :128])
    assert torch.equal(out[..., :128], want) and bool((out[..., 128:] == 2).all())
    same = ops.attend(pool, rows, c.q[:1].expand_as(c.q))  # a broadcast query
    assert torch.equal(same, ops.attend(pool, rows, c.q[:1].expand_as(c.q).contiguous()))
    q = c.q.clone()
    assert ops.attend(pool, rows, q, gate=c.gate, out=q) is q and torch.equal(q, want)
    g = c.gate.clone()
    assert torch.equal(ops.attend(pool, rows, c.q, gate=g, out=g), want)


def test_attend_is_deterministic_and_ignores_the_hint(ops):
    c = Case([(3, 5000), (1, 70), (150, 900)], 12, 2, 256, "q8", "f16", seed=14)
    pool, rows = c.ops()
    first = ops.attend(pool, rows, c.q)
    for _ in range(3):
        assert torch.equal(ops.attend(pool, rows, c.q)[:c.rows_used], first[:c.rows_used])
    want, bound = c.attend_ref()
    for hint in (0, 1, 10**6):
        rows = ops.KVRows(c.start, c.kv_len, c.tables, c.n_rows, hint)
        assert_within(ops.attend(pool, rows, c.q)[:c.rows_used], want, bound)


def test_many_sequences(ops):
    """Decoding batches: the most sequences a call takes, and one beyond."""
    from speculative_decode_persistent_gb300.mk import MkError
    c = Case([(1 + i % 3, 3 + (7 * i) % 50) for i in range(1024)], 4, 2, 64, "f16", "f16", seed=15)
    check_attend(ops, c)
    before = {n: t.clone() for n, t in c.pool.items()}
    pool, rows = c.ops()
    ops.kv_write(pool, rows, c.new_k, c.new_v)
    assert not torch.equal(bits(before["k"]), bits(c.pool["k"]))
    c = Case([(1, 1)] * 1025, 4, 2, 64, "f16", "f16")
    for fn in (lambda: ops.attend(*c.ops(), c.q), lambda: ops.kv_write(*c.ops(), c.new_k, c.new_v), lambda: ops.kv_read(*c.ops())):
        with pytest.raises(MkError) as e:
            fn()
        assert e.value.status == -8


def test_nothing_to_do(ops):
    c = Case([(0, 20), (0, 0)], 4, 2, 64, pad_rows=0)
    pool, rows = c.ops()
    assert ops.attend(pool, rows, c.q).shape == (0, 4, 64)
    assert ops.kv_read(pool, rows)[0].shape == (0, 2, 64)
    ops.kv_write(pool, rows, c.new_k, c.new_v)
    c = Case([(0, 20), (0, 0)], 4, 2, 64, pad_rows=3)  # rows, but of no sequence
    check_attend(ops, c)


# ----------------------------------------------------------- streams, graphs
def test_captured_and_replayed(ops):
    """Two graphs of the three operators, replayed in turn on changed lengths, pages and inputs."""
    c = Case([(2, 40), (130, 400)], 6, 1, 256, "q8", "f16", seed=16)
    pool, rows = c.ops()

    def once():
        ops.kv_write(pool, rows, c.new_k, c.new_v)
        return (ops.attend(pool, rows, c.q, window=50, sinks=4),) + ops.kv_read(pool, rows)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        once()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = once()
        graphs.append((g, out))
    for step in range(3):
        c.q.copy_(torch.randn_like(c.q))
        c.new_k.copy_(torch.randn_like(c.new_k))
        if step == 2:
            c.kv_len.copy_(torch.tensor([31, 385], dtype=torch.int32))
            c.tables.copy_(c.tables.flip(0))
            c.tables[0, 20], c.tables[1, 2] = c.tables[0, 1], -1
        for g, _ in graphs:
            g.replay()
        want = once()
        for g, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a[:c.rows_used], b[:c.rows_used])


def test_on_other_streams_at_once(ops):
    cases = [Case([(3, 3000 + 100 * i), (40, 200)], 12, 2, 256, ("f16", "q8")[i % 2], "f16", seed=20 + i) for i in range(4)]
    want = [ops.attend(*c.ops(), c.q) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(ops.attend(*c.ops(), c.q))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        c = cases[i % 4]
        assert torch.equal(g[:c.rows_used], want[i % 4][:c.rows_used])


def test_beyond_32_bit_offsets(ops):
    """A pool of more than 2^32 bytes and 2^31 elements whose last pages are in use."""
    n_pages, hkv, dh = (1 << 31) // (4 * 16 * 256) + 40, 4, 256
    small = Case([(3, 400), (2, 33)], 8, hkv, dh, "f16", "f16", seed=17)
    big = {n: torch.empty((n_pages, hkv, 16, dh), dtype=torch.float16, device="cuda") for n in ("k", "v")}
    off = n_pages - small.n_pages
    for n in big:
        big[n][off:] = small.pool[n]
    pool = ops.KVPool(big["k"], big["v"])
    tables = torch.where(small.tables >= 0, small.tables + off, small.tables)
    rows = ops.KVRows(small.start, small.kv_len, tables, small.n_rows, 3)
    want, bound = small.attend_ref()
    assert_within(ops.attend(pool, rows, small.q)[:5], want, bound)
    ops.kv_write(pool, rows, small.new_k, small.new_v)
    k, v = ops.kv_read(pool, rows)
    assert torch.equal(k[:5], small.new_k[:5]) and torch.equal(v[:5], small.new_v[:5])


# -------------------------------------------------------------- run together
def _f64(a):
    return np.asarray(a, np.float64)


@pytest.mark.parametrize("kv_q8", [0, 1])
def test_engine_context_written_read_and_attended(ops, kv_q8):
    """A sequence read from one engine with seq_kv and installed in another with seq_load decodes the
    same tokens; attend over the engine's pool equals the reference on it."""
    from gen.workload import Workload
    from speculative_decode_persistent_gb300 import mk
    wl = Workload("tiny", norm_jitter=0.1, overrides=dict(kv_q8=kv_q8))
    cached = wl.seqs[0][0]
    S, conv = wl.states[0]
    engines = [mk.Engine(wl.model, wl.weights, kv_q8, wl.n_pages) for _ in range(2)]
    engines[0].load_pool(wl.pool)
    engines[0].seq_set(0, cached, wl.tables[0], S, conv)
    k, v = engines[0].seq_kv(0, torch.float32)
    assert k.shape == (1, cached, wl.model["hkv"], wl.model["dh"])
    engines[1].seq_load(3, k[:, :5], v[:, :5])       # takes the lowest pages first
    engines[1].seq_load(0, k, v, S, conv)
    assert list(engines[1].seq_get(0)["pages"]) == [1, 2, 3, 4]
    k1, v1 = engines[1].seq_kv(0, torch.float32)
    if kv_q8:  # requantising code x scale gives the block again only up to the scale's rounding
        assert float((k1 - k).abs().max()) <= float(k.abs().max()) / 127
    else:
        assert torch.equal(k1, k) and torch.equal(v1, v)
        tok, pos, sid = wl.rows()
        assert [list(x) for x in engines[1].step(tok, pos, sid)] == [list(x) for x in engines[0].step(tok, pos, sid)]
        assert torch.equal(*[e.seq_kv(0)[0][:, :cached] for e in engines])
    for e in engines:
        e.commit([0], [1]) if not kv_q8 else None
    eng = engines[1]
    n = eng.seq_get(0)["length"]
    q = torch.randn((7 + 5, 4, 64), device="cuda").half()
    out = eng.attend(0, q, [0, 3], [7, 5], window=20, sinks=2)
    kk, vv = (torch.cat([eng.seq_kv(0, torch.float32)[i][0], eng.seq_kv(3, torch.float32)[i][0]]).double() for i in (0, 1))
    at, r = 0, 0
    for T, m in ((n, 7), (5, 5)):
        kx, vx = kk[at:at + T, 0], vv[at:at + T, 0]
        at += T
        t, p = torch.arange(T, device="cuda"), torch.arange(T - m, T, device="cuda")[:, None]
        see = (t <= p) & ((p - t < 20) | (t < 2))
        s = torch.einsum("nhd,td->nht", q[r:r + m].double(), kx) / 8
        w = torch.softmax(torch.where(see[:, None], s, -math.inf), -1)
        want = torch.einsum("nht,td->nhd", w, vx)
        assert float((out[r:r + m].double() - want).abs().max()) < 1e-2
        r += m
    for e in engines:
        e.close()


def test_engine_refusals(ops):
    from gen import configs
    from gen.synth import make_weights
    from speculative_decode_persistent_gb300 import mk
    eng = mk.Engine(configs.TINY, make_weights(configs.TINY, 0), 0, 4)
    z = lambda n: torch.zeros((1, n, 1, 64), device="cuda", dtype=torch.float16)  # noqa: E731
    eng.seq_load(0, z(40), z(40))
    for status, fn in ((-2, lambda: eng.seq_load(1, z(20), z(20))), (-1, lambda: eng.seq_load(8, z(1), z(1))),
                       (-1, lambda: eng.seq_load(1, z(1)[0], z(1)[0])), (-1, lambda: eng.kv_pool(1)),
                       (-1, lambda: eng.seq_load(1, z(1), z(1), S=np.zeros((3, 4, 64, 63), np.float32))),
                       (-1, lambda: eng.seq_rows([0], [41])), (-1, lambda: eng.attend(0, z(1)[0], [0], [1]))):
        with pytest.raises(mk.MkError) as e:
            fn()
        assert e.value.status == status
    assert eng.seq_get(0)["length"] == 40
    eng.close()


# -------------------------------------------- many blocks and items a worker
LONG = [([(5, 30000)], 12, 2, 256), ([(600, 9000), (1, 3000), (33, 33)], 12, 2, 128), ([(700, 20000)], 4, 1, 64),
        ([(300, 12000), (300, 300)], 6, 2, 192), ([(2000, 2000)], 6, 1, 256), ([(1, 1500)] * 200, 8, 4, 128),
        ([(40, 45)] * 300, 6, 3, 256)]


@pytest.mark.parametrize("kv,dtype", [("f16", "f16"), ("q8", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("seqs,hq,hkv,dh", LONG)
def test_attend_long(ops, seqs, hq, hkv, dh, kv, dtype):
    """Every worker takes many blocks, of one item and of many; run again and again the result is the same."""
    c = Case(seqs, hq, hkv, dh, kv, dtype, seed=30, pad_rows=0)
    out = check_attend(ops, c)
    pool, rows = c.ops()
    for _ in range(10):
        assert torch.equal(ops.attend(pool, rows, c.q), out)


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_attend_long_window(ops, kv):
    check_attend(ops, Case([(500, 20000), (3, 900), (1, 15000)], 12, 2, 256, kv, "bf16", seed=31), 1500, 40, gate=True)


def test_lengths_and_tables_of_any_value(ops):
    """Rows that run backwards, lengths and page ids out of range: nothing outside the buffers is
    touched, the call ends, and the next one is right."""
    c = Case([(9, 300), (70, 400), (1, 50)], 6, 2, 128, "q8", "f16", seed=32)
    pool, rows = c.ops()
    want = ops.attend(pool, rows, c.q)
    n = c.n_rows
    big = 2 ** 31 - 1
    for start in ([0, 9, 3, 80], [50, 20, 10, 0], [-5, 1000, 9, 70], [big, 0, -big, big]):
        for lens in ([300, -4, big], [-big, 0, 17]):
            t = c.tables.clone()
            t[0, ::2], t[1, 1::3] = big, -big
            r = ops.KVRows(torch.tensor(start, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           t, n, 70)
            out = torch.zeros((n + 4, 6, 128), dtype=torch.float16, device="cuda")
            ops.attend(pool, r, c.q, out=out[2:n + 2], window=30, sinks=2)
            k = torch.zeros((n + 4, 2, 128), dtype=torch.float16, device="cuda")
            ops.kv_read(pool, r, out=(k[2:n + 2], k.clone()[2:n + 2]))
            torch.cuda.synchronize()
            assert not out[:2].any() and not out[n + 2:].any() and not k[:2].any() and not k[n + 2:].any()
    assert torch.equal(ops.attend(pool, rows, c.q)[:c.rows_used], want[:c.rows_used])


def test_write_q8_infinities_and_nan_as_the_step_stores_them(ops):
    from speculative_decode_persistent_gb300 import mk
    x = torch.randn((64, 32), device="cuda")
    x[1, 3], x[2, 4], x[3, 5], x[4] = math.inf, -math.inf, math.nan, math.nan
    x[5] *= 8.3e6 / float(x[5].abs().max())        # a scale near binary16's largest value
    x[6] *= 9e6 / float(x[6].abs().max())          # and past it
    x[7] = 1e-9
    c = Case([(32, 32)], hkv=1, dh=64, kv="q8", dtype="f32", pad_rows=0)
    c.new_k.copy_(x.view(32, 1, 64))
    ops.kv_write(*c.ops(), c.new_k, c.new_k)
    q, d = mk.q8_encode(x)
    page = c.tables[0].long().repeat_interleave(16)[:32]
    slot = torch.arange(32, device="cuda") % 16
    assert torch.equal(c.pool["k"][page, 0, slot].reshape(64, 32), q)
    assert torch.equal(bits(c.pool["k_scale"][page, 0, slot]).reshape(64), d)


def test_first_call_inside_a_capture(tmp_path):
    """A process whose first calls are captured, and replayed."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = (
        "import sys, torch; sys.path[:0] = [%r, %r]\n" % (root, os.path.join(root, "tests")) +
        "from ops_helpers import Case, assert_within\n"
        "from speculative_decode_persistent_gb300 import ops\n"
        "c = Case([(3, 700), (150, 200)], 6, 2, 128, 'q8', 'f16', seed=3)\n"
        "pool, rows = c.ops(); g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    out = ops.attend(pool, rows, c.q); k, v = ops.kv_read(pool, rows)\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "assert_within(out[:153], *c.attend_ref()); assert torch.equal(k[:3], c.gather(0, 'k')[0][-3:].half()); print('same')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kv", ["f16", "q8"])
def test_sequences_that_share_pages(ops, kv):
    """A common prefix on the same pages, and one sequence twice."""
    c = Case([(4, 200), (150, 330), (1, 96)], 6, 2, 256, kv, "f16", seed=33)
    c.tables[0, :6], c.tables[2, :6] = c.tables[1, :6], c.tables[1, :6]
    out = check_attend(ops, c)
    pool, rows = c.ops()
    twice = ops.KVRows(torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"), c.kv_len[:1].repeat(2), c.tables[:1].repeat(2, 1), 8)
    got = ops.attend(pool, twice, c.q[:4].repeat(2, 1, 1))
    assert torch.equal(got[:4], got[4:])
    assert float((got[:4].double() - out[:4].double()).abs().max()) < 2e-3  # (cut elsewhere)
    k, v = ops.kv_read(pool, rows, torch.float32)
    for i, (n, T) in enumerate(c.seqs):
        r = int(c.start[i])
        assert torch.equal(k[r:r + n], c.gather(i, "k")[0][T - n:].float())


def test_engine_loads_nothing_and_goes_on(ops):
    """An empty context is an empty sequence: the same tokens as after seq_new."""
    from gen import configs
    from gen.synth import make_weights
    from speculative_decode_persistent_gb300 import mk
    eng = mk.Engine(configs.TINY, make_weights(configs.TINY, 0), 0, 16)
    z = torch.zeros((1, 0, 1, 64), device="cuda", dtype=torch.float16)
    eng.seq_load(0, z, z)
    eng.seq_new(1)
    got = [list(eng.step([5, 6, 7], [0, 1, 2], [s] * 3, [1, 1, 2])[0]) for s in (0, 1)]
    assert got[0] == got[1] and eng.seq_get(0)["length"] == 3
    k, v = eng.seq_kv(0)
    k1, v1 = eng.seq_kv(1)
    # (split sums are added in any order: a rounding apart)
    assert torch.allclose(k.float(), k1.float(), atol=1e-3) and torch.allclose(v.float(), v1.float(), atol=1e-3)
    eng.close()
