"""Cases, plain forms and costs of the operators for trees of drafted tokens.

Per sequence, the last q of its n cached tokens are the nodes of a tree: node
j's parent is a node before it, or none (-1: it follows the cached tokens
before the tree). A node's slot in the cache is n - q + j, its position n - q +
its depth. On a paged pool ([layers][pages][kv heads][16 tokens][head dim],
binary16, or 8-bit codes with one binary16 scale per 32 dims):

rope    normalises q and k per head (optional gains), rotates them by the rows'
        positions, and stores k and v in the pool (rounded, or quantised);
attend  attention of each node over the cached tokens and its own ancestors;
accept  greedy verification: the path of nodes that the logits agree with;
keep    moves the kept nodes' K and V, in all layers, up to the slots behind
        the cached tokens, and gives the new lengths; also drops old tokens;
copy    copies pages in all layers, so that a prefix serves another sequence.

A case's `seqs` lists its sequences as "new rows @ cached tokens, the new rows
among them". `kv` is the pool's type, `dtype` the type of the dense tensors.
"""
import math

import torch

own = False

PAGE = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BASE, EPS = 1e7, 1e-6


def listed():
    heads = {"hq": 24, "hkv": 4, "dh": 256}
    small = {"hq": 4, "hkv": 1, "dh": 64}
    full = {"window": 0, "sinks": 0, "gate": False}
    return [
        # one agent drafts a small tree over a 4K context: the smallest verify pass
        {"name": "attend-tree8-4k-f16", "op": "attend", "kv": "f16", "dtype": "bf16", "seqs": "8@4104", **full, **heads},
        # four agents' trees of 16 nodes over 23K quantised tokens each, with the model's output gate
        {"name": "attend-4xtree16-23k-q8", "op": "attend", "kv": "q8", "dtype": "bf16", "seqs": ",".join(["16@23016"] * 4),
         "window": 0, "sinks": 0, "gate": True, **heads},
        # a tree of 64 nodes deep in a long context
        {"name": "attend-tree64-96k-f16", "op": "attend", "kv": "f16", "dtype": "bf16", "seqs": "64@96064", **full, **heads},
        # a ragged batch of trees, one of a single node and one with nothing cached, small heads, window and sinks
        {"name": "attend-ragged-dh64-f16", "op": "attend", "kv": "f16", "dtype": "f16", "seqs": "1@65,13@68,37@3001,21@21",
         "window": 512, "sinks": 4, "gate": False, **small},
        # four agents' trees enter a quantised cache, q and k normalised
        {"name": "rope-4xtree16-q8", "op": "rope", "kv": "q8", "dtype": "bf16", "seqs": ",".join(["16@23016"] * 4), "rot": 256,
         "norm": True, **heads},
        # a whole prompt
        {"name": "rope-prompt8k-f16", "op": "rope", "kv": "f16", "dtype": "bf16", "seqs": "8192@8192", "rot": 64, "norm": True,
         **heads},
        # verification of one agent's small tree, a small vocabulary
        {"name": "accept-tree8-v2k", "op": "accept", "dtype": "f32", "seqs": "8@4104", "vocab": 2048},
        # four agents' trees of 16 nodes, the full vocabulary
        {"name": "accept-4xtree16-v248k", "op": "accept", "dtype": "f32", "seqs": ",".join(["16@23016"] * 4), "vocab": 248320},
        # the accepted paths of four trees move up, in all 17 layers
        {"name": "keep-4xtree16-17layers-f16", "op": "keep", "kv": "f16", "seqs": ",".join(["16@1040"] * 4), "kept": "5,2,1,4",
         "sinks": 0, "layers": 17, "hkv": 4, "dh": 256},
        # a 23K context loses its middle: 16 first and 8,176 last tokens stay
        {"name": "keep-evict-23k-17layers-q8", "op": "keep", "kv": "q8", "seqs": "23000@23000", "kept": "8192", "sinks": 16,
         "layers": 17, "hkv": 4, "dh": 256},
        # a conversation is forked: its last, partly filled page, in all layers
        {"name": "copy-1page-17layers-q8", "op": "copy", "kv": "q8", "pages": 1, "ways": 1, "layers": 17, "hkv": 4, "dh": 256},
        # a prefix of 4K tokens is given to three more agents
        {"name": "copy-3x4k-17layers-f16", "op": "copy", "kv": "f16", "pages": 256, "ways": 3, "layers": 17, "hkv": 4, "dh": 256},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "rope", "rope", "accept", "keep", "copy"))
    case = {"op": op}
    if op == "accept":
        n = rng.choice((1, 2, 3, 4, 8))
        case["dtype"] = rng.choice(("f32", "f16", "bf16"))
        case["vocab"] = _log(rng, 100, 248320)
        most = 64 * 248320 // case["vocab"]  # the largest listed case's logits
        seqs = [(min(rng.choice((1, rng.randint(2, 16), rng.randint(17, 128))), max(1, most // n)), 0) for _ in range(n)]
        case["seqs"] = ",".join("%d@%d" % (q, q + rng.randint(0, 500)) for q, _ in seqs)
        return case
    dh = rng.choice((64, 128, 192, 256, 256))
    hkv = rng.choice((1, 2, 3, 4, 8) if dh < 256 else (1, 2, 4))
    case |= {"kv": rng.choice(("f16", "q8")), "hkv": hkv, "dh": dh}
    if op == "copy":
        case["layers"], case["ways"] = rng.choice((1, 2, 5, 16, 17)), rng.choice((1, 1, 2, 3))
        case["pages"] = _log(rng, 1, max(1, 17 * 256 * 1024 // (case["layers"] * hkv * dh)))
        return case
    if op == "keep":
        case["layers"] = rng.choice((1, 2, 5, 16, 17))
        if rng.random() < 0.3:  # old tokens are dropped
            n = _log(rng, 20, max(20, 17 * 23000 * 1024 // (case["layers"] * hkv * dh) // (2 if case["kv"] == "f16" else 1)))
            n = min(n, 90000)
            case["sinks"] = rng.choice((0, 4, rng.randint(1, 9)))
            kept = max(1, rng.randint(1, n) // 2 - 2 * case["sinks"]) + case["sinks"]
            case |= {"seqs": "%d@%d" % (n, n), "kept": str(kept)}
            return case
        n = rng.choice((1, 2, 3, 4, 8))
        q = [rng.choice((1, rng.randint(2, 16), rng.randint(17, 128))) for _ in range(n)]
        case |= {"sinks": 0, "seqs": ",".join("%d@%d" % (x, x + _log(rng, 1, 3000)) for x in q),
                 "kept": ",".join(str(rng.randint(1, max(1, x // 2))) for x in q)}
        return case
    n = rng.choice((1, 1, 2, 3, 4, 8))
    case["hq"] = hkv * rng.choice((1, 2, 3, 4, 6, 8) if hkv <= 4 else (1, 2, 4))
    if op == "rope":
        case |= {"dtype": rng.choice(("f16", "bf16", "f32") if case["kv"] == "f16" else ("f16", "bf16")),
                 "rot": rng.choice([x for x in (64, 128, 192, 256) if x <= dh]), "norm": rng.choice((True, True, False))}
        most = int(8192 * 32 * 256 * 2 / ((case["hq"] + 2 * hkv) * dh * TYPES[case["dtype"]].itemsize))
        q = [max(1, min(rng.choice((1, rng.randint(2, 64), _log(rng, 1, 8192))), most // n)) for _ in range(n)]
        case["seqs"] = ",".join("%d@%d" % (x, x + _log(rng, 1, 40000 // n) - 1) for x in q)
        return case
    case["dtype"] = rng.choice(("f16", "bf16"))
    seqs = []
    for _ in range(n):
        t = _log(rng, 1, 90000 // n)
        q = rng.choice((1, rng.randint(2, 16), rng.randint(17, 64), rng.randint(65, 256)))
        q = max(1, min(q, int(1.5e11 / (n * 4 * case["hq"] * dh * t))))  # the largest listed case's operations
        seqs.append((q, t + q - 1))
    case["window"] = rng.choice((0, 0, 0, _log(rng, 1, 8000)))
    case["sinks"] = rng.choice((0, 4, rng.randint(1, 300))) if case["window"] else 0
    case["gate"] = rng.choice((False, True))
    case["seqs"] = ",".join("%d@%d" % s for s in seqs)
    return case


def _seqs(case):
    return [tuple(int(x) for x in s.split("@")) for s in case["seqs"].split(",")]


def _pool(state, g, layers, n_pages):
    case = state["case"]
    shape = (n_pages, case["hkv"], PAGE, case["dh"])
    if layers:
        shape = (layers,) + shape
    for name in ("k", "v"):
        state[name + "_scale"] = None
        if case["kv"] == "f16":
            state[name] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
        else:
            blocks = shape[:-1] + (shape[-1] // 32,)
            state[name] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
            state[name + "_scale"] = (torch.rand(blocks, generator=g, device="cuda") * 0.01 + 0.015).half()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "copy":
        n, ways = case["pages"], case["ways"]
        n_pages = n * (1 + ways) + 2
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        _pool(state, g, case["layers"], n_pages)
        state["src"], state["dst"] = order[:n].repeat(ways), order[n:n * (1 + ways)].contiguous()
        return state
    seqs = _seqs(case)
    pages = [-(-kv // PAGE) for _, kv in seqs]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(seqs), max(pages)), -1, dtype=torch.int32, device="cuda")
    at, start = 0, [0]
    for i, n in enumerate(pages):
        tables[i, :n] = order[at:at + n]
        at += n
        start.append(start[-1] + seqs[i][0])
    rows = start[-1]
    state |= {"tables": tables, "n_rows": rows, "max_q": max(q for q, _ in seqs), "row_start": i32(start),
              "kv_len": i32([kv for _, kv in seqs])}
    j = torch.cat([torch.arange(q, device="cuda") for q, _ in seqs])
    # a random tree: any earlier node may be the parent (a prompt is a chain)
    parents = (j * rand(rows)).floor().clamp_max(j - 1)
    state["parents"] = torch.where(j == 0, -1, parents).to(torch.int32)
    if case["op"] == "accept":
        state["tokens"] = (rand(rows) * case["vocab"]).long().clamp_max(case["vocab"] - 1).to(torch.int32)
        x = torch.randn(rows, case["vocab"], generator=g, device="cuda")
        # the model agrees with most drafts that continue a text it likes
        first = state["row_start"][:-1].long().repeat_interleave(i32([q for q, _ in seqs]))
        child = ((j > 0) & (rand(rows) < 0.7)).nonzero()[:, 0]
        x[first[child] + state["parents"][child].long(), state["tokens"][child].long()] = 6 + rand(len(child))
        state["logits"] = x.to(TYPES[case["dtype"]])
        return state
    _pool(state, g, case.get("layers", 0), n_pages)
    if case["op"] == "keep":
        # ascending nodes; those that move lie behind the slots that they move to, so that a pass can be repeated
        keep = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        for i, kept in enumerate(int(x) for x in case["kept"].split(",")):
            q, stay = seqs[i][0], max(1, case["sinks"])
            stay = min(stay, kept)
            if case["sinks"] or q == seqs[i][1]:
                moved = torch.arange(q - (kept - stay), q, device="cuda")
            else:
                moved = (kept + torch.randperm(q - kept, generator=g, device="cuda")[:kept - stay]).sort().values
            keep[start[i]:start[i] + kept] = torch.cat([torch.arange(stay, device="cuda"), moved]).to(torch.int32)
        state["keep"] = keep
        return state
    dt = TYPES[case["dtype"]]
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    if case["op"] == "rope":
        qkv = torch.randn(rows, hq + 2 * hkv, dh, generator=g, device="cuda").to(dt)  # one projection's output
        state["q"], state["new_k"], state["new_v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        for name in ("q_gain", "k_gain"):
            state[name] = 0.5 + rand(dh) if case["norm"] else None
        if max(q for q, _ in seqs) > 256:
            state["parents"] = None
        return state
    state["q"] = torch.randn(rows, hq, dh, generator=g, device="cuda").to(dt)
    state["gate"] = torch.randn(rows, hq, dh, generator=g, device="cuda").to(dt) if case["gate"] else None
    return state


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def _own(state):
    from speculative_decode_persistent_gb300 import ops
    case, pool = state["case"], (state["k"], state["v"], state["k_scale"], state["v_scale"]) if "k" in state else None
    if case["op"] == "copy":
        ops.kv_copy(ops.KVLayers(*pool), state["src"], state["dst"])
        return _words(state)
    rows = ops.KVRows(state["row_start"], state["kv_len"], state["tables"], state["n_rows"], state["max_q"])
    if case["op"] == "attend":
        return ops.attend(ops.KVPool(*pool), rows, state["q"], window=case["window"], sinks=case["sinks"], gate=state["gate"],
                          parents=state["parents"])
    if case["op"] == "accept":
        return ops.tree_accept(rows, state["parents"], state["tokens"], state["logits"])
    if case["op"] == "keep":
        return _words(state) + (ops.kv_keep(ops.KVLayers(*pool), rows, state["keep"]),)
    if "rope" not in state:  # kept, as a program keeps it for all of its calls
        state["rope"] = ops.Rope(case["rot"], BASE, state["q_gain"], state["k_gain"], EPS, device="cuda")
    pool = ops.KVPool(*pool)
    q = ops.rope_write(pool, rows, state["rope"], state["q"], state["new_k"], state["new_v"], parents=state["parents"])
    return (q, state["k"], state["v"]) if case["kv"] == "f16" else (q,) + ops.kv_read(pool, rows, TYPES[case["dtype"]])


def _words(state):
    """A pool that was only moved about: its values, or the words of memory that hold its codes and scales."""
    if state["k_scale"] is None:
        return state["k"], state["v"]
    return tuple(state[n].view(torch.int32) for n in ("k", "v")) + tuple(state[n + "_scale"].view(torch.int16) for n in ("k", "v"))


# ------------------------------------------------------------- plain forms
def _rows(state):
    """(sequence, index within it) of every row."""
    row, start = torch.arange(state["n_rows"], device="cuda"), state["row_start"].long()
    seq = (row[:, None] >= start[None, 1:]).sum(1)
    return seq, row - start[seq]


def _base(state):
    """Cached tokens before each sequence's new rows."""
    start = state["row_start"].long()
    return state["kv_len"].long() - (start[1:] - start[:-1])


def _double(a):
    return (a @ a).clamp_max(1)


def _lineage(state):
    """[sequences][node][node]: whether the second is the first or one of its ancestors, in 32 bits."""
    (seq, j), m = _rows(state), state["max_q"]
    a = torch.eye(m, device="cuda").repeat(len(state["kv_len"]), 1, 1)
    p = state["parents"].long()
    a[seq, j, torch.where(p < 0, j, p)] = 1
    return _double(_double(_double(_double(_double(_double(_double(_double(a))))))))


def _plain_copy(state):
    src, dst = state["src"].long(), state["dst"].long()
    state["k"][:, dst], state["v"][:, dst] = state["k"][:, src], state["v"][:, src]
    if state["k_scale"] is not None:
        state["k_scale"][:, dst], state["v_scale"][:, dst] = state["k_scale"][:, src], state["v_scale"][:, src]
    return _words(state)


def _plain_keep(state):
    seq, j = _rows(state)
    base, keep = _base(state), state["keep"].long()
    to = base[seq] + j
    at = torch.where(keep < 0, to, base[seq] + keep)  # slots that nothing moves to stay what they are
    page, slot = state["tables"][seq, to // PAGE].long(), to % PAGE
    page0, slot0 = state["tables"][seq, at // PAGE].long(), at % PAGE
    state["k"][:, page, :, slot], state["v"][:, page, :, slot] = state["k"][:, page0, :, slot0], state["v"][:, page0, :, slot0]
    if state["k_scale"] is not None:
        state["k_scale"][:, page, :, slot] = state["k_scale"][:, page0, :, slot0]
        state["v_scale"][:, page, :, slot] = state["v_scale"][:, page0, :, slot0]
    count = torch.zeros_like(base).index_add_(0, seq, (keep >= 0).long())
    return _words(state) + ((base + count).to(torch.int32),)


def _plain_accept(state):
    (seq, j), m, vocab = _rows(state), state["max_q"], state["case"]["vocab"]
    logits = state["logits"].float()
    top = logits.amax(-1, keepdim=True)
    greedy = torch.where(logits == top, torch.arange(vocab, device="cuda"), vocab).amin(-1)  # the first of the largest
    first = state["row_start"].long()[seq]
    parent, tok = first + state["parents"].long().clamp_min(0), state["tokens"].long()
    good = (j > 0) & (state["parents"] >= 0) & (tok == greedy[parent])
    # of several good children of a node the first
    rival = (parent[:, None] == parent) & good[:, None] & good & (j[:, None] > j)
    good = (good & ~rival.any(1)) | (j == 0)
    bad = torch.ones(len(state["kv_len"]), m, device="cuda")
    bad[seq, j] = 1 - good.float()
    lineage = _lineage(state)
    on = (lineage @ bad[..., None])[seq, j, 0] == 0  # the node and all of its ancestors
    on &= lineage[seq, j, 0] == 1
    place = torch.cumsum(on, 0) - 1
    count = torch.zeros(len(state["kv_len"]), dtype=torch.long, device="cuda").index_add_(0, seq, on.long())
    place = first + place - (torch.cumsum(count, 0) - count)[seq]
    path = torch.full((state["n_rows"] + 1,), -1, device="cuda")
    emitted = path.clone()
    place = torch.where(on, place, state["n_rows"])
    path[place], emitted[place] = j, greedy
    return path[:-1].to(torch.int32), count.to(torch.int32), emitted[:-1].to(torch.int32)


def _half(x):
    """A positive 64-bit value rounded once to the nearest binary16 (ties to even), as a 64-bit value."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -30))).clamp_min(-14) - 10)
    return torch.round(x / step) * step


def _store(state, name, page, slot, x):
    if state["case"]["kv"] == "f16":
        state[name][page, :, slot] = x.to(torch.float16)
        return
    x = x.double().unflatten(-1, (-1, 32))  # 64 bits: the quotients next to a rounding border
    d = _half(x.abs().amax(-1) / 127)
    c = torch.where(d[..., None] > 0, torch.round(x / d[..., None]).clamp(-127, 127), 0.0)
    state[name][page, :, slot] = c.flatten(-2).to(torch.int8)
    state[name + "_scale"][page, :, slot] = d.to(torch.float16)


def _load(state, name, page, slot):
    x = state[name][page, :, slot].float().unflatten(-1, (-1, 32))
    return (x * state[name + "_scale"][page, :, slot].float()[..., None]).flatten(-2).to(TYPES[state["case"]["dtype"]])


def _plain_rope(state):
    case, (seq, j) = state["case"], _rows(state)
    half, base = case["rot"] // 2, _base(state)
    slot = base[seq] + j
    pos = slot if state["parents"] is None else base[seq] + (_lineage(state).sum(-1).long() - 1)[seq, j]
    # 64 bits: the angles of far positions
    a = pos[:, None].double() * BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
        lo, hi = x[..., :half], x[..., half:2 * half]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, x[..., 2 * half:]], -1)

    q = turned(state["q"], state["q_gain"]).to(state["q"].dtype)
    page, slot = state["tables"][seq, slot // PAGE].long(), slot % PAGE
    _store(state, "k", page, slot, turned(state["new_k"], state["k_gain"]))
    _store(state, "v", page, slot, state["new_v"].float())
    if case["kv"] == "f16":
        return q, state["k"], state["v"]
    return q, _load(state, "k", page, slot), _load(state, "v", page, slot)


def _context(state, name):
    """Every sequence's cached rows, padded to the longest: [sequences][kv heads][tokens][head dim] in 32 bits."""
    t = state["tables"].long().clamp_min(0)
    x = state[name][t].float()
    if state["case"]["kv"] == "q8":
        x = (x.unflatten(-1, (-1, 32)) * state[name + "_scale"][t].float()[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(state):
    case, q, (seq, j) = state["case"], state["q"], _rows(state)
    hkv, dh, m = case["hkv"], case["dh"], state["max_q"]
    k, v, base = _context(state, "k"), _context(state, "v"), _base(state)
    n, _, toks, _ = k.shape
    qp = torch.zeros(n, m, case["hq"], dh, device="cuda")
    qp[seq, j] = q.float()
    qp = qp.unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [n][hkv][nodes][group][dh]
    s = torch.matmul(qp.flatten(2, 3), k.transpose(-1, -2)).mul_(1 / math.sqrt(dh)).view(n, hkv, m, -1, toks)
    lineage = _lineage(state)
    depth = lineage.sum(-1).long() - 1
    # tokens as nodes of the tree: [n][nodes][tokens]
    node = torch.arange(toks, device="cuda") - base[:, None]
    cached, at = node < 0, node.clamp(0, m - 1)
    seen = cached[:, None] | (lineage.gather(2, at[:, None].expand(n, m, toks)) > 0)
    seen &= (node < m)[:, None]
    if case["window"]:
        pos = torch.where(cached, node, depth.gather(1, at))  # behind the cached tokens
        near = depth[:, :, None] - pos[:, None] < case["window"]
        seen &= near | (pos + base[:, None] < case["sinks"])[:, None]
    seen = seen[:, None, :, None]
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.flatten(2, 3), v).view(n, hkv, m, -1, dh)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, j]
    if state["gate"] is not None:
        o = o / (1 + torch.exp(-state["gate"].float()))
    return o.to(q.dtype)


PLAIN = {"copy": _plain_copy, "keep": _plain_keep, "accept": _plain_accept, "rope": _plain_rope, "attend": _plain_attend}


# -------------------------------------------------------------------- cost
def work(case):
    item = 2 if case.get("kv") == "f16" else 1 + 2 / 32
    if case["op"] == "copy":  # each source page in once, each copy out
        return {"bytes": (1 + case["ways"]) * case["pages"] * case["layers"] * case["hkv"] * PAGE * case["dh"] * 2 * item,
                "flops": 0}
    seqs = _seqs(case)
    rows = sum(q for q, _ in seqs)
    if case["op"] == "accept":
        return {"bytes": rows * (case["vocab"] * TYPES[case["dtype"]].itemsize + 16), "flops": 0}
    if case["op"] == "keep":  # the tokens that move, in and out
        kept = [int(x) for x in case["kept"].split(",")]
        moved = sum(k - min(k, max(1, case["sinks"])) for k in kept)
        return {"bytes": moved * case["layers"] * case["hkv"] * case["dh"] * 2 * item * 2 + 4 * sum(kept), "flops": 0}
    hq, hkv, dh, wide = case["hq"], case["hkv"], case["dh"], TYPES[case["dtype"]].itemsize
    if case["op"] == "rope":  # q in and out, k and v in and to the pool; quantised rows read back
        back = 2 * hkv * (item + wide) if case["kv"] == "q8" else 0
        return {"bytes": rows * dh * (2 * hq * wide + 2 * hkv * (wide + item) + back), "flops": 0}
    # at least the cached tokens before the tree (those in the window) and the node itself
    w = case["window"] or 1 << 40
    seen = [(q, min(kv - q, w - 1) + 1) for q, kv in seqs]
    cache = sum(t + q - 1 for q, t in seen) * hkv * dh * 2 * item
    return {"bytes": cache + rows * (hq * dh * wide * (3 if case["gate"] else 2) + 4),
            "flops": 4 * hq * dh * sum(q * t for q, t in seen)}


# ---------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"copy": _exact_copy, "keep": _exact_keep, "accept": _exact_accept, "rope": _exact_rope,
            "attend": _exact_attend}[case["op"]](case, state)


def _exact_words(state, move):
    out = []
    for n in ("k", "v", "k_scale", "v_scale"):
        if state[n] is not None:
            t = move(state[n].clone())
            out.append(t.double() if state["k_scale"] is None else t.view(torch.int32 if len(n) == 1 else torch.int16))
    return out


def _exact_copy(case, state):
    src, dst = state["src"].tolist(), state["dst"].tolist()

    def move(t):
        was = t.clone()
        for a, b in zip(src, dst):
            t[:, b] = was[:, a]
        return t
    return tuple(_exact_words(state, move))


def _exact_keep(case, state):
    lengths, pairs, at = [], [], 0
    for i, (q, kv) in enumerate(_seqs(case)):
        keep = [x for x in state["keep"][at:at + q].tolist() if x >= 0]
        table = state["tables"][i].tolist()
        pairs += [(table[(kv - q + x) // PAGE] * PAGE + (kv - q + x) % PAGE, table[(kv - q + y) // PAGE] * PAGE + (kv - q + y) % PAGE)
                  for y, x in enumerate(keep)]
        lengths.append(kv - q + len(keep))
        at += q
    a, b = torch.tensor(pairs, device="cuda").T

    def move(t):  # by token: [layers][tokens of all pages][kv heads][dims]
        flat = t.transpose(2, 3).flatten(1, 2)
        flat[:, b] = flat[:, a]
        return flat.unflatten(1, (-1, PAGE)).transpose(2, 3).contiguous()
    return tuple(_exact_words(state, move)) + (torch.tensor(lengths, dtype=torch.int32),)


def _exact_accept(case, state):
    logits, tok, par = state["logits"].double().cpu().numpy(), state["tokens"].tolist(), state["parents"].tolist()
    path, emitted, counts, at = [], [], [], 0
    for q, _ in _seqs(case):
        kids = {}
        for j in range(1, q):
            kids.setdefault(par[at + j], []).append(j)
        walk, out, cur = [], [], 0
        while cur is not None:
            walk.append(cur)
            out.append(int(logits[at + cur].argmax()))  # the first of the largest
            cur = next((c for c in kids.get(cur, []) if tok[at + c] == out[-1]), None)
        counts.append(len(walk))
        path += walk + [-1] * (q - len(walk))
        emitted += out + [-1] * (q - len(walk))
        at += q
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (path, counts, emitted))


def _ancestors(parents):
    """Each node's ancestors and itself, of one tree."""
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else []) + [j])
    return out


def _exact_rope(case, state):
    rot, pos, rows, at = case["rot"], [], [], 0
    for i, (q, kv) in enumerate(_seqs(case)):
        line = None if state["parents"] is None else _ancestors(state["parents"][at:at + q].tolist())
        pos += [kv - q + (j if line is None else len(line[j]) - 1) for j in range(q)]
        rows += [(i, kv - q + j) for j in range(q)]
        at += q
    freq = torch.tensor([BASE ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(torch.tensor(pos, device="cuda").double(), freq))

    def turned(x, gain):
        x = x.to(torch.float64)
        if gain is not None:
            x = x / ((x * x).mean(dim=-1, keepdim=True) + EPS).sqrt() * gain.to(torch.float64)
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn[:, None, :]
        return torch.cat((z.real, z.imag, x[..., rot:]), dim=-1)

    q = turned(state["q"], state["q_gain"])
    new = turned(state["new_k"], state["k_gain"]), state["new_v"].to(torch.float64)
    if case["kv"] == "q8":
        return (q,) + tuple(_quantised(x) for x in new)
    seq, slot = torch.tensor(rows, device="cuda").T
    out = []
    for name, x in zip("kv", new):
        t = state[name].to(torch.float64)
        t[state["tables"][seq, slot.div(PAGE, rounding_mode="floor")].long(), :, slot.remainder(PAGE)] = x
        out.append(t)
    return (q,) + tuple(out)


def _quantised(x):
    """What an 8-bit cache holds of x: 32 values share the scale amax / 127, kept in 16 bits."""
    b = x.reshape(-1, 32)
    d = (b.abs().max(dim=1, keepdim=True).values / 127).to(torch.float32).to(torch.float16).to(torch.float64)
    return (torch.round(b / d).clip(-127, 127) * d).reshape(x.shape)


def _exact_attend(case, state):
    hkv, dh, out, at = case["hkv"], case["dh"], [], 0
    for i, (n, kv) in enumerate(_seqs(case)):
        line = _ancestors(state["parents"][at:at + n].tolist())
        base, w = kv - n, case["window"]
        see = torch.zeros(n, kv, dtype=torch.bool)
        see[:, :base] = True
        for j, nodes in enumerate(line):
            where = base + len(nodes) - 1
            if w:
                see[j, :max(0, min(base, where - w + 1))] = False
                see[j, :min(base, case["sinks"])] = True
            for depth, x in enumerate(nodes):
                see[j, base + x] = not w or len(nodes) - 1 - depth < w or base + depth < case["sinks"]
        see = see.to("cuda")
        pages = state["tables"][i, :-(-kv // PAGE)].long()
        x = {}
        for name in ("k", "v"):
            t = state[name][pages].to(torch.float64)
            if case["kv"] == "q8":
                t = t * state[name + "_scale"][pages].to(torch.float64).repeat_interleave(32, dim=-1)
            x[name] = t.permute(1, 0, 2, 3).reshape(hkv, -1, dh)[:, :kv]
        q = state["q"][at:at + n].to(torch.float64).reshape(n, hkv, -1, dh)
        at += n
        by_head = []
        for h in range(hkv):
            s = torch.einsum("ngd,td->gnt", q[:, h], x["k"][h]) / dh ** 0.5
            p = torch.softmax(s.masked_fill_(~see, -math.inf), dim=-1)
            by_head.append(torch.einsum("gnt,td->ngd", p, x["v"][h]))
            del s, p
        out.append(torch.stack(by_head, 1).reshape(n, -1, dh))
    o = torch.cat(out)
    return o if state["gate"] is None else o * torch.sigmoid(state["gate"].to(torch.float64))
