"""Calls of the KV-cache operators around the GPU work: outputs in other layouts, errors that another
call left, contexts loaded into an engine, the engine's own stream, waits that give up."""
import os
import sys

import numpy as np
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


def _tiny(**kw):
    from gen import configs
    from gen.synth import make_weights
    from speculative_decode_persistent_gb300 import mk
    return mk.Engine(configs.TINY, make_weights(configs.TINY, 0), 0, 16, **kw)


def test_an_error_that_another_call_left(ops):
    """The runtime's last error, left by an unrelated host call, is neither reported nor cleared by the
    calls that are queued after it."""
    from speculative_decode_persistent_gb300 import mk
    c = Case([(3, 20)], 4, 2, 64, "q8", "f16", seed=51, pad_rows=0)
    pool, rows = c.ops()
    x = torch.randn((4, 32), device="cuda")
    calls = (lambda: ops.kv_write(pool, rows, c.new_k, c.new_v), lambda: ops.kv_read(pool, rows),
             lambda: ops.attend(pool, rows, c.q), lambda: mk.q8_encode(x))
    for call in calls:
        call()
    torch.cuda.synchronize()
    host = torch.empty(64)
    for call in calls:
        assert int(torch.cuda.cudart().cudaHostUnregister(host.data_ptr())) != 0  # it was never registered
        call()
        with pytest.raises(RuntimeError):  # still there, for the next check of torch's own
            torch.ones(3, device="cuda")
        torch.cuda.synchronize()
    k, _ = ops.kv_read(pool, rows)
    assert float((k.float() - c.new_k.float()).abs().max()) < 0.05


def _decode(eng, seq, n):
    """n greedy tokens of a sequence, one row a step, each step's token fed into the next."""
    got, token = [], 11
    for _ in range(n):
        out, _ = eng.step([token], [eng.seq_get(seq)["length"]], [seq])
        eng.commit([seq], [1])
        token = int(out[0])
        got.append(token)
    return got


def test_a_context_saved_and_loaded_again(ops):
    """What seq_kv and seq_get give is what seq_load takes: K, V and the recurrent state, on the device or
    from the host."""
    eng = _tiny()
    eng.seq_new(0)
    eng.step([5, 6, 7, 8], [0, 1, 2, 3], [0] * 4, [1, 1, 1, 2])
    info, (k, v) = eng.seq_get(0), eng.seq_kv(0)
    assert info["length"] == 4 and k.shape[1] == 4
    S, conv = info["S"].clone(), info["conv"].clone()
    eng.seq_load(1, k, v, info["S"], info["conv"])
    eng.seq_load(2, k, v, S.cpu().numpy(), conv.double())
    eng.seq_load(3, k, v, S.cpu(), conv.cpu().numpy())
    for s in (1, 2, 3):
        now = eng.seq_get(s)
        assert now["length"] == 4 and torch.equal(now["S"], S) and torch.equal(now["conv"], conv)
        assert all(torch.equal(a, b) for a, b in zip(eng.seq_kv(s), (k, v)))
    want = _decode(eng, 0, 5)
    assert all(_decode(eng, s, 5) == want for s in (1, 2, 3))
    eng.close()


def test_a_refused_load_leaves_the_old_context(ops):
    from speculative_decode_persistent_gb300.mk import MkError
    eng = _tiny()
    eng.seq_new(0)
    eng.step([5, 6, 7, 8], [0, 1, 2, 3], [0] * 4, [1, 1, 1, 2])
    eng.seq_load(0, *eng.seq_kv(0), eng.seq_get(0)["S"], eng.seq_get(0)["conv"])  # state in slot 0 now
    info, (k, v) = eng.seq_get(0), eng.seq_kv(0)
    S, conv, pages = info["S"].clone(), info["conv"].clone(), list(info["pages"])
    other = torch.randn_like(k)
    words = np.full(tuple(S.shape), "x")
    for status, args in ((-1, (other, other, words)), (-1, (other, other, S * 2, np.full(tuple(conv.shape), "x"))),
                         (-1, (other, other, None, conv[1:])), (-1, (other, other, S * 2, conv[..., 1:])), (-1, (other, other, S[None])),
                         (-1, (other.double(), other.double())), (-1, (other, other.float())), (-1, (other, other.cpu())),
                         (-1, (other, other[:, :2])), (-1, (torch.randn((1, 16 * 16 + 1, 1, 64), device="cuda"),) * 2)):
        with pytest.raises(MkError) as e:
            eng.seq_load(0, *args)
        assert e.value.status == status
        now = eng.seq_get(0)
        assert now["length"] == 4 and list(now["pages"]) == pages
        assert torch.equal(now["S"], S) and torch.equal(now["conv"], conv)
        assert all(torch.equal(a, b) for a, b in zip(eng.seq_kv(0), (k, v)))
    eng.close()


def test_calls_on_another_stream_come_after_the_engines_work(ops):
    """The engine on a stream of its own, the calls on the default one: they see what was queued there
    before, and what they write is not overtaken by it."""
    s = torch.cuda.Stream()
    eng = _tiny(stream=s)
    one = lambda x: torch.full((1, 40, 1, 64), x, device="cuda", dtype=torch.float16)  # noqa: E731
    eng.seq_load(0, one(1.0), one(1.0))
    half = torch.float16

    def later(x):  # the pool's values change on the engine's stream, a tenth of a second from now
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)
            for t in eng.kv_views().values():
                t.view(half).fill_(x)

    later(2.0)
    assert all(bool((t == 2).all()) for t in eng.seq_kv(0))
    q = torch.zeros((3, 4, 64), device="cuda", dtype=half)
    later(3.0)
    assert bool((eng.attend(0, q, [0], [3]) == 3).all())
    later(4.0)
    eng.seq_load(0, one(5.0), one(5.0))
    assert all(bool((t == 5).all()) for t in eng.seq_kv(0))
    eng.close()


# (workers that have blocks: an item's 4 or 8 first units of the line have none, with few items a worker may get only such)
@pytest.mark.parametrize("kv,seqs,hq,hkv,dh,skip,large", [
    ("f16", [(3, 3000), (1, 500)], 6, 2, 128, 15, False), ("f16", [(300, 2000), (2, 60)], 6, 2, 256, 4, False),
    ("q8", [(3, 5000)], 6, 2, 256, 20, False), ("q8", [(150, 900), (1, 400)], 12, 2, 256, 5, False),
    ("q8", [(1, 300)] * 200, 4, 2, 64, 5, False), ("q8", [(3, 3000)] * 3, 6, 2, 256, 40, True), ("q8", [(150, 900)] * 8, 12, 2, 128, 3, True)])
def test_a_wait_that_gives_up(ops, kv, seqs, hq, hkv, dh, skip, large):
    """One worker's queries are never handed over: its waits run out after 2 ms, its rows become NaN, all
    others are right, the call ends and so does the next one, with the right result."""
    c = Case(seqs, hq, hkv, dh, kv, "bf16", seed=60, amp=2e5 if large else 1.0)
    kw = dict(scale=1.0 / (2e5 * dh ** 0.5)) if large else {}
    pool, rows = c.ops()
    want, bound = c.attend_ref(**kw)
    before = ops.attend(pool, rows, c.q, **kw)[:c.rows_used]
    assert_within(before, want, bound)
    assert [ops.lib.mk_debug_attend_wait(*x) for x in ((-1, -1), (2_000_001, -1), (0, -2))] == [-1] * 3
    assert ops.lib.mk_debug_attend_wait(2_000, skip) == 0
    try:
        for _ in range(2):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            got = ops.attend(pool, rows, c.q, **kw)[:c.rows_used]
            b.record()
            torch.cuda.synchronize()
            lost = torch.isnan(got).all(-1)
            assert bool(lost.any()) and not bool(lost.all())
            assert_within(got[~lost], want[~lost], bound[~lost])
            assert a.elapsed_time(b) < 1000.0
    finally:
        ops.lib.mk_debug_attend_wait(0, -1)
    assert torch.equal(ops.attend(pool, rows, c.q, **kw)[:c.rows_used], before)
