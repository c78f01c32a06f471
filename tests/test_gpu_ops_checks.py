"""Refusals of the pool operators' Python calls with CUDA tensors: the tested argument is the only fault, the
message names it, and nothing is written. And acceptance of trees larger than a block's shared memory."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops(request):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_persistent_gb300 import ops as o
    return o


def h(*s):
    return torch.ones(s, dtype=torch.float16, device="cuda")


def i(*s):
    return torch.ones(s, dtype=torch.int32, device="cuda")


def test_refused_calls(ops):
    N = 5
    k0, v0 = h(4, 2, 16, 64), h(4, 2, 16, 64)
    pool = ops.KVPool(k0, v0)
    start, length, tables = torch.tensor([0, N], dtype=torch.int32, device="cuda"), i(1) * 40, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    rows = ops.KVRows(start, length, tables, n_rows=N)
    cpu_rows = ops.KVRows(start.cpu(), length.cpu(), tables.cpu(), n_rows=N)
    q, k, lg = h(N, 4, 64), h(N, 2, 64), torch.ones(N, 7, device="cuda")
    out = h(N, 4, 64) * 7
    rope = ops.Rope(64, device="cuda")
    gains = torch.ones(128, device="cuda")
    lk, lv = h(3, 4, 2, 16, 64), h(3, 4, 2, 16, 64)
    layers, cpu_layers = ops.KVLayers(lk, lv), ops.KVLayers(lk.cpu(), lv.cpu())
    rw = lambda **kw: lambda: ops.rope_write(pool, rows, kw.pop("rope", rope), q, k, k, out=out, **kw)  # noqa: E731
    at = lambda **kw: lambda: ops.attend(pool, rows, q, out=out, **kw)  # noqa: E731
    ta = lambda p=i(N), t=i(N), x=lg, r=rows: lambda: ops.tree_accept(r, p, t, x)  # noqa: E731
    cp = lambda s=i(3), d=i(3), x=layers: lambda: ops.kv_copy(x, s, d)  # noqa: E731
    kp = lambda e=i(N), r=rows, x=layers: lambda: ops.kv_keep(x, r, e)  # noqa: E731
    bad_index = [i(N - 1), i(N + 1), i(0), i(N).long(), i(N).float(), i(N).cpu(), i(2 * N)[::2], i(N, 1), i(1).expand(N)]
    cases = []
    for x in bad_index:
        cases += [(at(parents=x), "attend parents"), (rw(parents=x), "rope_write parents"), (rw(positions=x), "rope_write positions"),
                  (ta(p=x), "tree_accept parents"), (ta(t=x), "tree_accept tokens")]
        cases += [(kp(x), "kv_keep")]
    for x in (i(2), i(4), i(3).long(), i(3).cpu(), i(6)[::2], i(3, 1)):
        cases += [(cp(d=x), "kv_copy dst")]
    for x in (i(3).long(), i(3).cpu(), i(6)[::2], i(3, 1)):
        cases += [(cp(s=x), "kv_copy")]
    cases += [
        (ta(t=None), "tokens"), (ta(p="x"), "(a tensor)"), (ta(x=lg.cpu()), "one CUDA device"), (ta(r=cpu_rows), "one CUDA device"),
        (ta(x=lg[:4]), "rows of the logits"), (ta(x=torch.ones(7, N, device="cuda").t()), "logits [rows]"),
        (cp(x=cpu_layers), "a CUDA device"), (kp(x=cpu_layers), "one CUDA device"), (kp(r=cpu_rows), "one CUDA device"),
        (rw(parents=i(N), positions=i(N)), "parents or positions"), (rw(rope=ops.Rope(64, device="cpu")), "Rope on the pool's device"),
        (rw(rope=ops.Rope(128, device="cuda")), "no more dims"), (rw(rope=ops.Rope(64, q_gain=gains)), "gains for all"),
        (lambda: ops.rope_write(pool, rows, rope, q, k, k.cpu(), out=out), "one CUDA device"),
        (lambda: ops.rope_write(pool, cpu_rows, rope, q, k, k, out=out), "one CUDA device"),
        (lambda: ops.rope_write(pool, rows, rope, q, k, k, out=out.cpu()), "one CUDA device"),
        (lambda: ops.rope_write(pool, rows, rope, q, k, k[:4], out=out), "one number of rows"),
        (lambda: ops.rope_write(pool, rows, rope, q.requires_grad_(), k, k, out=out), "no gradient"),
        (lambda: ops.rope_write(pool, rows, rope, q.detach(), k, k, out=out[:1].expand(N, 4, 64)), "must not overlap"),
        (lambda: ops.attend(pool, rows, q.detach(), out=out[:1].expand(N, 4, 64)), "must not overlap"),
        (lambda: ops.attend(pool, rows, h(N, 3, 64), out=out[:, :3]), "mk_attend"), (at(window=-1), "a window"), (at(scale=0.0), "positive scale"),
        (at(sinks=2), "mk_attend"), (lambda: ops.attend(pool, rows, q.detach(), out=out, gate=h(N, 4, 64).cpu()), "one CUDA device"),
        (lambda: ops.kv_write(pool, rows, k, k[:4]), "one number of rows"), (lambda: ops.kv_write(pool, rows, k, k.cpu()), "one CUDA device"),
        (lambda: ops.kv_read(pool, rows, out=(k, k.float())), "of one type"), (lambda: ops.kv_read(pool, cpu_rows, torch.float16), "one CUDA device")]
    for n, (call, says) in enumerate(cases):
        q = q.detach() if n else q
        with pytest.raises(ops.MkError) as e:
            call()
        assert e.value.status == -1 and says in str(e.value), (n, says, str(e.value))
    torch.cuda.synchronize()
    for t in (k0, v0, lk, lv, k):
        assert bool((t == 1).all())
    assert bool((out == 7).all())


@pytest.mark.parametrize("nodes,vocab", [(1500, 50), (1025, 3), (2600, 300)])
def test_accepted_paths_beyond_a_blocks_memory(ops, nodes, vocab):
    """A path that goes past the 1,024 nodes whose greedy tokens a block keeps in shared memory, in a chain and through
    every other node of a tree, beside a small sequence."""
    from test_gpu_tree_ops import check_accept
    g = torch.Generator().manual_seed(nodes)
    for step in (1, 2):
        line = list(range(0, nodes, step))  # the nodes that the model agrees with; the others are leaves that it does not
        parents = [j - step if j % step == 0 else j - 1 for j in range(nodes)]
        tok = torch.randint(0, vocab, (nodes + 3,), generator=g, dtype=torch.int32)
        if step == 2:
            tok[1:nodes - 1:2] = (tok[2:nodes:2][:len(tok[1:nodes - 1:2])] + 1) % vocab
        x = torch.zeros(nodes + 3, vocab)
        for a, c in zip(line, line[1:]):
            x[a, tok[c]] = 1.0
        x[line[-1], (tok[nodes - 1] + 1) % vocab] = 1.0  # (a last leaf)
        assert check_accept(ops, [nodes, 3], parents + [-1, 0, 1], tok.cuda(), x.cuda()) == len(line)
    # only the last node disagrees
    tok = torch.arange(nodes, dtype=torch.int32) % vocab
    x = torch.zeros(nodes, vocab)
    x[torch.arange(nodes - 1), tok[1:].long()] = 1.0
    x[nodes - 2] = 0.0
    x[nodes - 2, (int(tok[nodes - 1]) + 1) % vocab] = 1.0
    assert check_accept(ops, [nodes], list(range(-1, nodes - 1)), tok.cuda(), x.cuda(), pass_parents=False) == nodes - 1
