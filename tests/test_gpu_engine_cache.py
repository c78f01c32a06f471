"""An engine's cached contexts copied and thinned out (Engine.clone_sequence, seq_keep): models without KV
layers, the recurrent state of what is kept, calls beside the engine's own stream."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.fixture(scope="module")
def mk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import mk as m
    return m


def _engine(mk, kinds=None, **kw):
    from gen import configs
    from gen.synth import make_weights
    model = dict(configs.TINY, **({} if kinds is None else {"kinds": kinds}))
    return mk.Engine(model, make_weights(model, 0), 0, 16, **kw)


def _decode(eng, seq, n, token=11):
    got = []
    for _ in range(n):
        out, _ = eng.step([token], [eng.seq_get(seq)["length"]], [seq])
        eng.commit([seq], [1])
        token = int(out[0])
        got.append(token)
    return got


def test_models_without_kv_layers(mk):
    """Recurrent layers only: a sequence has pages and a state, and no layer keeps K and V."""
    eng = _engine(mk, [0, 0, 0, 0])
    eng.seq_new(0)
    for i, t in enumerate((5, 6, 7)):
        eng.step([t], [i], [0])
        eng.commit([0], [1])
    eng.clone_sequence(0, 1)
    a, b = eng.seq_get(0), eng.seq_get(1)
    assert b["length"] == a["length"] == 3 and torch.equal(a["S"], b["S"]) and torch.equal(a["conv"], b["conv"])
    eng.clone_sequence(1, 1)
    assert eng.seq_keep(1, 2, [0]) == 2 and eng.seq_get(1)["length"] == 2
    assert eng.seq_keep(1, 0, []) == 2
    eng.clone_sequence(0, 1)
    assert _decode(eng, 0, 4) == _decode(eng, 1, 4)
    eng.close()


def test_copies_come_after_the_engines_work(mk):
    """The engine on a stream of its own, the calls on the default one: the states that they copy are those that the
    work queued there leaves, also where no K and V move."""
    s = torch.cuda.Stream()
    eng = _engine(mk, stream=s)
    eng.seq_new(0)
    eng.step([5, 6, 7, 8], [0, 1, 2, 3], [0] * 4, [1, 1, 1, 2])
    assert eng.seq_get(0)["slot"] != 0

    def later(seq, x):  # the committed state changes on the engine's stream, a tenth of a second from now
        slot = eng.seq_get(seq)["slot"]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)
            for t in eng.state_views():
                t[seq, slot].fill_(x)

    def all_are(seq, x):
        info = eng.seq_get(seq)
        return info["slot"] == 0 and bool((info["S"] == x).all()) and bool((info["conv"] == x).all())

    later(0, 2.0)
    assert eng.seq_keep(0, 0, []) == 4 and all_are(0, 2.0)
    later(0, 3.0)
    eng.clone_sequence(0, 0)
    assert eng.seq_get(0)["length"] == 4 and all_are(0, 3.0)
    later(0, 4.0)
    eng.clone_sequence(0, 1)
    assert all_are(1, 4.0)
    S, conv = (torch.full_like(eng.seq_get(1)[x], 6.0) for x in ("S", "conv"))
    later(1, 7.0)
    eng.seq_set(1, 4, eng.seq_get(1)["pages"], S, conv)
    assert all_are(1, 6.0)
    later(1, 8.0)
    eng.seq_new(1)
    assert all_are(1, 0.0)
    eng.seq_new(2)  # nothing cached: no pages to copy either
    later(2, 5.0)
    eng.clone_sequence(2, 3)
    assert eng.seq_get(3)["length"] == 0 and all_are(3, 5.0)
    eng.close()


def test_kept_tokens_with_their_state(mk):
    """After rejected tokens the state of the kept ones goes in with them, and the sequence goes on as one that never
    saw the others."""
    eng = _engine(mk)
    want = None
    for seq, texts in ((0, (5, 6)), (1, (5, 6, 7, 8))):
        eng.seq_new(seq)
        for i, t in enumerate(texts):
            eng.step([t], [i], [seq])
            eng.commit([seq], [1])
            if i == 1:
                S, conv = (eng.seq_get(seq)[x].clone() for x in ("S", "conv"))
        if seq == 0:
            eng.clone_sequence(0, 2)
            eng.clone_sequence(0, 3)
            want = _decode(eng, 0, 6)
    assert eng.seq_keep(1, 2, [], S, conv) == 2
    assert torch.equal(eng.seq_get(1)["S"], S) and torch.equal(eng.seq_get(1)["conv"], conv)
    assert _decode(eng, 1, 6) == want
    # the second of two drafts beside each other was right: its K and V lie one slot too far, its state is given from the host
    eng.step([9], [2], [2])
    eng.commit([2], [1])
    eng.step([9], [2], [3])
    eng.commit([3], [1])
    S, conv = eng.seq_get(3)["S"].cpu(), eng.seq_get(3)["conv"].cpu().numpy()
    k, v = eng.seq_kv(2)
    eng.seq_load(4, torch.cat([k[:, :2], k[:, 1:2], k[:, 2:]], 1), torch.cat([v[:, :2], v[:, 1:2], v[:, 2:]], 1))
    assert eng.seq_keep(4, 2, [1], S, conv) == 3
    assert all(torch.equal(a, b) for a, b in zip(eng.seq_kv(4), (k, v)))
    assert _decode(eng, 4, 6) == _decode(eng, 3, 6)
    eng.close()


def test_a_refused_keep_leaves_everything(mk):
    eng = _engine(mk)
    eng.seq_new(0)
    eng.step([5, 6, 7, 8], [0, 1, 2, 3], [0] * 4, [1, 1, 1, 2])
    info, (k, v) = eng.seq_get(0), eng.seq_kv(0)
    S, conv = info["S"].clone(), info["conv"].clone()
    for args in ((5, [0]), (2, [2]), (2, [1, 0]), (2, [0], S[None]), (2, [0], S, conv[1:]), (2, [0], "x"), (2, [0], S, [["x"]])):
        with pytest.raises(mk.MkError) as e:
            eng.seq_keep(0, *args)
        assert e.value.status == -1
        now = eng.seq_get(0)
        assert now["length"] == 4 and torch.equal(now["S"], S) and torch.equal(now["conv"], conv)
        assert all(torch.equal(a, b) for a, b in zip(eng.seq_kv(0), (k, v)))
    # one of the two alone: the other stays
    assert eng.seq_keep(0, 1, [], None, conv * 2) == 3
    assert torch.equal(eng.seq_get(0)["S"], S) and torch.equal(eng.seq_get(0)["conv"], conv * 2)
    eng.close()


def test_a_sequence_that_there_is_not(mk):
    """A number below 0 would index the last sequence's state from behind: refused before anything is written."""
    eng = _engine(mk)
    last = eng.max_seqs - 1
    for s in (0, last):
        eng.seq_new(s)
        eng.step([5 + s], [0], [s])
        eng.commit([s], [1])
    eng.clone_sequence(last, last)  # state in slot 0
    before = [eng.seq_get(last)[x].clone() for x in ("S", "conv")]
    k = eng.seq_kv(0)
    for seq in (-1, -last - 1, eng.max_seqs):
        for call in (lambda: eng.seq_set(seq, 0, [], before[0] * 2, before[1] * 2), lambda: eng.seq_new(seq), lambda: eng.clone_sequence(0, seq),
                     lambda: eng.seq_load(seq, *k), lambda: eng.seq_keep(seq, 0, []), lambda: eng.clone_sequence(seq, 0)):
            with pytest.raises(mk.MkError) as e:
                call()
            assert e.value.status == -1
    now = eng.seq_get(last)
    assert torch.equal(now["S"], before[0]) and torch.equal(now["conv"], before[1])
    eng.close()
