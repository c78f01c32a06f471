"""Cases, plain forms and costs of the paged KV-cache operators.

Three operators on one layer of a paged pool ([pages][kv heads][16 tokens][head
dim], binary16, or 8-bit codes with one binary16 scale per 32 dims):

write   stores new rows of K and V at the end of their sequences (rounded, or
        quantised) and reads the rows back as the values the pool now stands for;
read    gathers the rows of whole contexts back into dense tensors;
attend  causal attention of each sequence's new rows over its cached tokens,
        with grouped heads, an optional sliding window whose first `sinks`
        tokens stay visible, and an optional sigmoid output gate.

A case's `seqs` lists its sequences as "new rows @ cached tokens, the new rows
among them". `kv` is the pool's type, `dtype` the type of the dense tensors.
"""
import math

import torch

own = False

PAGE = 16
F32 = torch.float32
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    big = {"hkv": 4, "dh": 256}
    heads = {"hq": 24, "hkv": 4, "dh": 256}
    return [
        # one new token of one sequence enters an fp16 cache: the smallest call
        {"name": "write-f16-1", "op": "write", "kv": "f16", "dtype": "bf16", "seqs": "1@4097", **big},
        # the verify rows of four agents (4 x 3) enter a quantised cache
        {"name": "write-q8-4x3", "op": "write", "kv": "q8", "dtype": "f32", "seqs": "3@23003,3@23003,3@23003,3@23003", **big},
        # one prompt chunk
        {"name": "write-q8-chunk512", "op": "write", "kv": "q8", "dtype": "bf16", "seqs": "512@20512", **big},
        # four whole contexts, computed elsewhere, are installed at once
        {"name": "write-q8-4x23k", "op": "write", "kv": "q8", "dtype": "bf16",
         "seqs": "23000@23000,23000@23000,23000@23000,23000@23000", **big},
        # short conversations of odd lengths are saved, small heads
        {"name": "read-q8-odd", "op": "read", "kv": "q8", "dtype": "f32", "seqs": "37@37,1@1,1003@1003", "hkv": 1, "dh": 64},
        # one long context is read back
        {"name": "read-f16-96k", "op": "read", "kv": "f16", "dtype": "bf16", "seqs": "96000@96000", **big},
        # plain decoding: one token over a 4K cache
        {"name": "attend-t1-4k-f16", "op": "attend", "kv": "f16", "dtype": "bf16", "seqs": "1@4097", "window": 0, "sinks": 0,
         "gate": False, **heads},
        # four agents' verify rows over 23K quantised tokens each
        {"name": "attend-4x3-23k-q8", "op": "attend", "kv": "q8", "dtype": "bf16",
         "seqs": "3@23003,3@23003,3@23003,3@23003", "window": 0, "sinks": 0, "gate": True, **heads},
        # one prompt chunk deep in a quantised context
        {"name": "attend-chunk512-20k-q8", "op": "attend", "kv": "q8", "dtype": "bf16", "seqs": "512@20512", "window": 0,
         "sinks": 0, "gate": False, **heads},
        # a whole prompt at once: the compute-bound end
        {"name": "attend-prompt4k-f16", "op": "attend", "kv": "f16", "dtype": "f16", "seqs": "4096@4096", "window": 0,
         "sinks": 0, "gate": False, **heads},
        # a chunk of a long document with a window and its first tokens kept
        {"name": "attend-window4k-96k-f16", "op": "attend", "kv": "f16", "dtype": "bf16", "seqs": "512@96512",
         "window": 4096, "sinks": 16, "gate": True, **heads},
        # a ragged batch of decoding, verify and prompt rows, small heads
        {"name": "attend-ragged-dh64-f16", "op": "attend", "kv": "f16", "dtype": "f16", "seqs": "1@65,4@68,117@301,64@64",
         "window": 0, "sinks": 0, "gate": False, "hq": 4, "hkv": 1, "dh": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend"))
    dh = rng.choice((64, 128, 192, 256, 256))
    hkv = rng.choice((1, 2, 3, 4, 8) if dh < 256 else (1, 2, 4))
    case = {"op": op, "kv": rng.choice(("f16", "q8")), "hkv": hkv, "dh": dh}
    n = rng.choice((1, 1, 2, 3, 4, 8))
    if op != "attend":
        case["dtype"] = rng.choice(("f16", "bf16", "f32"))
        most = int(1.1e9 / (2 * hkv * dh * (2 * TYPES[case["dtype"]].itemsize + 4)))  # the largest listed case's bytes
        lens = [_log(rng, 1, min(92000, most) // n) for _ in range(n)]
        seqs = [(t, t) for t in lens] if op == "read" else [(_log(rng, 1, t), t) for t in lens]
        case["seqs"] = ",".join("%d@%d" % s for s in seqs)
        return case
    case["hq"] = hkv * rng.choice((1, 2, 3, 4, 6, 8) if hkv <= 4 else (1, 2, 4))
    case["dtype"] = rng.choice(("f16", "bf16"))
    seqs = []
    for _ in range(n):
        t = _log(rng, 1, 40000 // n)
        # decoding, verify rows of a few drafts, or a chunk of a prompt
        q = rng.choice((1, rng.randint(2, 8), _log(rng, 9, 2000)))
        most = int(2e11 / (n * 4 * case["hq"] * dh * t))  # the largest listed case's operations
        seqs.append((min(q, t, most), t))
    case["window"] = rng.choice((0, 0, _log(rng, 1, 8000)))
    case["sinks"] = rng.choice((0, 4, rng.randint(1, 300))) if case["window"] else 0
    case["gate"] = rng.choice((False, True))
    case["seqs"] = ",".join("%d@%d" % s for s in seqs)
    return case


def _seqs(case):
    return [tuple(int(x) for x in s.split("@")) for s in case["seqs"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    seqs, hkv, dh = _seqs(case), case["hkv"], case["dh"]
    dt = TYPES[case["dtype"]]
    pages = [-(-kv // PAGE) for _, kv in seqs]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(seqs), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(pages):
        tables[i, :n] = order[at:at + n]
        at += n
    rows = sum(q for q, _ in seqs)
    state = {"case": case, "tables": tables, "n_rows": rows, "max_q": max(q for q, _ in seqs),
             "row_start": torch.tensor([0] + [sum(q for q, _ in seqs[:i + 1]) for i in range(len(seqs))],
                                       dtype=torch.int32, device="cuda"),
             "kv_len": torch.tensor([kv for _, kv in seqs], dtype=torch.int32, device="cuda")}
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    for name in ("k", "v"):
        x = rand(n_pages, hkv, PAGE, dh)
        state[name + "_scale"] = None
        if case["kv"] == "f16":
            state[name] = x.half()
        else:
            d = (x.view(n_pages, hkv, PAGE, dh // 32, 32).abs().amax(-1) / 127).half()
            state[name] = (x / d.float().repeat_interleave(32, -1)).round().clamp(-127, 127).to(torch.int8)
            state[name + "_scale"] = d
        del x
    if case["op"] == "write":
        state["new_k"], state["new_v"] = rand(rows, hkv, dh).to(dt), rand(rows, hkv, dh).to(dt)
    if case["op"] == "attend":
        state["q"] = rand(rows, case["hq"], dh).to(dt)
        state["gate"] = rand(rows, case["hq"], dh).to(dt) if case["gate"] else None
    return state


def run(state):
    case = state["case"]
    dt = TYPES[case["dtype"]]
    if own:
        from speculative_decode_persistent_gb300 import ops
        pool = ops.KVPool(state["k"], state["v"], state["k_scale"], state["v_scale"])
        rows = ops.KVRows(state["row_start"], state["kv_len"], state["tables"], state["n_rows"], state["max_q"])
        if case["op"] == "write":
            ops.kv_write(pool, rows, state["new_k"], state["new_v"])
            return ops.kv_read(pool, rows, dt)
        if case["op"] == "read":
            return ops.kv_read(pool, rows, dt)
        return ops.attend(pool, rows, state["q"], window=case["window"], sinks=case["sinks"], gate=state["gate"])
    if case["op"] == "attend":
        return _attend(state)
    page, slot = _places(state)
    if case["op"] == "write":
        _store(state, "k", page, slot, state["new_k"])
        _store(state, "v", page, slot, state["new_v"])
    return _load(state, "k", page, slot).to(dt), _load(state, "v", page, slot).to(dt)


# ------------------------------------------------------------- plain forms
def _places(state):
    """Page and slot of every row."""
    row = torch.arange(state["n_rows"], device="cuda")
    start, kv = state["row_start"].long(), state["kv_len"].long()
    seq = (row[:, None] >= start[None, 1:]).sum(1)
    pos = kv[seq] - start[seq + 1] + row
    return state["tables"][seq, pos // PAGE].long(), pos % PAGE


def _half(x):
    """A positive 64-bit value rounded once to the nearest binary16 (ties to even), as a 64-bit value."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -30))).clamp_min(-14) - 10)
    return torch.round(x / step) * step


def _store(state, name, page, slot, x):
    if _is_f16(state):
        state[name][page, :, slot] = x.to(torch.float16)
        return
    rows, hkv, dh = x.shape
    x = x.double().view(rows, hkv, dh // 32, 32)  # 64 bits: the quotients next to a rounding border
    d = _half(x.abs().amax(-1) / 127)
    c = torch.where(d[..., None] > 0, torch.round(x / d[..., None]).clamp(-127, 127), 0.0)
    state[name][page, :, slot] = c.view(rows, hkv, dh).to(torch.int8)
    state[name + "_scale"][page, :, slot] = d.to(torch.float16)


def _load(state, name, page, slot):
    x = state[name][page, :, slot].float()
    if _is_f16(state):
        return x
    return (x.unflatten(-1, (-1, 32)) * state[name + "_scale"][page, :, slot].float()[..., None]).flatten(-2)


def _is_f16(state):
    return state["case"]["kv"] == "f16"


def _context(state, name):
    """Every sequence's cached rows, padded to the longest: [sequences][kv heads][tokens][head dim] in 32 bits."""
    t = state["tables"].long().clamp_min(0)
    x = state[name][t].float()
    if not _is_f16(state):
        x = (x.unflatten(-1, (-1, 32)) * state[name + "_scale"][t].float()[..., None]).flatten(-2)
    return x.transpose(1, 2).flatten(2, 3)


def _attend(state):
    case, q = state["case"], state["q"]
    hkv, dh = case["hkv"], case["dh"]
    start, kv = state["row_start"].long(), state["kv_len"].long()
    k, v = _context(state, "k"), _context(state, "v")
    n, _, toks, _ = k.shape
    # new rows, padded to the longest sequence's: [sequences][rows]
    j = torch.arange(state["max_q"], device="cuda")
    q_len = start[1:] - start[:-1]
    qp = q.float()[(start[:-1, None] + j).clamp_max(q.shape[0] - 1)]
    qp = qp.unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [n][hkv][rows][group][dh]
    s = torch.matmul(qp.flatten(2, 3), k.transpose(-1, -2)).mul_(1 / math.sqrt(dh))
    s = s.view(n, hkv, state["max_q"], -1, toks)
    t = torch.arange(toks, device="cuda")
    pos = (kv - q_len)[:, None] + j
    seen = t <= pos[..., None]
    if case["window"]:
        seen &= (pos[..., None] - t < case["window"]) | (t < case["sinks"])
    seen = seen[:, None, :, None, :]
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.flatten(2, 3), v).view(n, hkv, state["max_q"], -1, dh)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n][rows][hq][dh]
    row = torch.arange(q.shape[0], device="cuda")
    seq = (row[:, None] >= start[None, 1:]).sum(1)
    o = o[seq, row - start[seq]]
    if state["gate"] is not None:
        o = o / (1 + torch.exp(-state["gate"].float()))
    return o.to(q.dtype)


# -------------------------------------------------------------------- cost
def _pairs(q, kv, window, sinks):
    """(row, token) pairs that see each other, and the tokens that some row sees."""
    first, pairs = kv - q, 0
    if not window:
        return q * first + q * (q + 1) // 2, kv
    for p in range(first, kv):
        pairs += min(window, p + 1) + max(0, min(sinks, p + 1 - window))
    low = max(0, first - window + 1)
    return pairs, kv - low + min(sinks, low)


def work(case):
    hkv, dh, seqs = case["hkv"], case["dh"], _seqs(case)
    item = 2 if case["kv"] == "f16" else 1 + 2 / 32
    wide = TYPES[case["dtype"]].itemsize
    rows = sum(q for q, _ in seqs)
    if case["op"] == "write":  # new rows in, the pool's rows out, and both again to read them back
        return {"bytes": 2 * rows * hkv * dh * (2 * wide + 2 * item), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * rows * hkv * dh * (item + wide), "flops": 0}
    both = [_pairs(q, kv, case["window"], case["sinks"]) for q, kv in seqs]
    cache = sum(t for _, t in both) * hkv * dh * 2 * item
    return {"bytes": cache + rows * case["hq"] * dh * wide * (3 if case["gate"] else 2),
            "flops": 4 * case["hq"] * dh * sum(p for p, _ in both)}


# ---------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    seqs, hkv, dh = _seqs(case), case["hkv"], case["dh"]
    value = {}
    for name in ("k", "v"):
        x = state[name].to(torch.float64)
        if case["kv"] == "q8":
            x = x * state[name + "_scale"].to(torch.float64).repeat_interleave(32, dim=-1)
        value[name] = x

    def tokens(name, i):  # the i-th sequence's cached rows: [tokens][kv heads][dh]
        x = value[name][state["tables"][i, :-(-seqs[i][1] // PAGE)].long()]
        return x.permute(0, 2, 1, 3).reshape(-1, hkv, dh)[:seqs[i][1]]

    if case["op"] == "read":
        return tuple(torch.cat([tokens(n, i) for i in range(len(seqs))]) for n in ("k", "v"))
    if case["op"] == "write":
        return tuple(_kept(state["new_" + n], case["kv"]) for n in ("k", "v"))
    out, at = [], 0
    for i, (n, kv) in enumerate(seqs):
        k, v = tokens("k", i), tokens("v", i)
        q = state["q"][at:at + n].to(torch.float64).reshape(n, hkv, -1, dh)
        at += n
        p = torch.arange(kv - n, kv, device=q.device).reshape(1, n, 1)
        t = torch.arange(kv, device=q.device)
        hide = t > p
        if case["window"]:
            hide |= (t <= p - case["window"]) & (t >= case["sinks"])
        by_head = []
        for h in range(hkv):
            s = torch.einsum("ngd,td->gnt", q[:, h], k[:, h]) / dh ** 0.5
            w = torch.softmax(s.masked_fill_(hide, -math.inf), dim=-1)
            by_head.append(torch.einsum("gnt,td->ngd", w, v[:, h]))
            del s, w
        out.append(torch.stack(by_head, 1).reshape(n, -1, dh))
    o = torch.cat(out)
    return o if state["gate"] is None else o * torch.sigmoid(state["gate"].to(torch.float64))


def _kept(x, kv):
    """What a cache of this type holds of x."""
    x = x.to(torch.float64)
    if kv == "f16":
        return _nearest_half(x)
    b = x.reshape(-1, 32)
    d = _nearest_half(b.abs().max(dim=1, keepdim=True).values / 127)
    c = torch.div(b, d)
    low = torch.floor(c)
    rest = c - low
    c = low + ((rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2) == 1)))
    return torch.nan_to_num(c.clip(-127, 127) * d, nan=0.0).reshape(x.shape)


def _nearest_half(x):
    """The nearest binary16 of each value, by its two neighbours' distances; the even one where they are equal."""
    h = x.to(torch.float32).to(torch.float16)
    bits = h.view(torch.int16).to(torch.int32)
    best, gap = h.to(torch.float64), (h.to(torch.float64) - x).abs()
    for step in (-1, 1):
        other = (bits + step).clamp(-32768, 32767).to(torch.int16).view(torch.float16).to(torch.float64)
        far = torch.nan_to_num((other - x).abs(), nan=math.inf)
        take = (far < gap) | ((far == gap) & (bits % 2 != 0))
        take &= torch.sign(other) * torch.sign(x) >= 0
        best, gap = torch.where(take, other, best), torch.where(take, far, gap)
    return best
