"""Cases and a 64-bit reference for the KV-cache operators.

The reference works token by token index on the pool's raw arrays, in double,
and shares no code with the package. `bound` is the elementwise error that the
kernel's documented roundings allow (derived below), not a measured value."""
import math

import torch

NP = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def q8_values(x):
    """(codes, scales) of x [..., n x 32] by the codec's definition, in double."""
    b = x.double().unflatten(-1, (-1, 32))
    d = half_even(b.abs().amax(-1) / 127)
    c = torch.where(d[..., None] > 0, torch.round(b / d[..., None]).clamp(-127, 127), torch.zeros((), dtype=torch.double, device=x.device))
    return c.flatten(-2), d


def half_even(x):
    """Nearest binary16 of non-negative doubles, ties to even (no double rounding)."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -40))).clamp_min(-14.0) - 10)
    return torch.round(x / step) * step


class Case:
    """A pool whose unused slots hold NaN, shuffled page tables and new rows."""

    def __init__(self, seqs, hq=4, hkv=2, dh=64, kv="f16", dtype="f16", seed=0, pad_rows=2, spare=3, device="cuda", amp=1.0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.dh, self.kv = seqs, hq, hkv, dh, kv
        self.dtype = NP[dtype]
        pages = [-(-t // 16) for _, t in seqs]
        self.n_pages = sum(pages) + spare
        order = torch.randperm(self.n_pages, generator=g).int()
        tables = torch.full((len(seqs), max(pages + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(pages):
            tables[i, :n] = order[at:at + n]
            at += n
        self.rows_used = sum(q for q, _ in seqs)
        self.n_rows = self.rows_used + pad_rows
        start = [0]
        for q, _ in seqs:
            start.append(start[-1] + q)
        self.tables = tables.to(device)
        self.start = torch.tensor(start, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([t for _, t in seqs], dtype=torch.int32, device=device)
        used = torch.zeros(self.n_pages, 1, 16, 1, dtype=torch.bool)
        for i, (_, t) in enumerate(seqs):
            for p in range(pages[i]):
                used[tables[i, p], 0, :max(0, t - 16 * p)] = True
        shape = (self.n_pages, hkv, 16, dh)
        self.pool, self.value = {}, {}
        for n in ("k", "v"):
            x = (torch.randn(shape, generator=g) * amp).to(device)
            u = used.to(device)
            if kv == "f16":
                h = torch.where(u, x, math.nan).half()
                self.pool[n] = h
                self.value[n] = h.double()
            else:
                c, d = q8_values(x)
                d = torch.where(u[..., :1].expand(shape[:3] + (dh // 32,)), d, math.nan).half()
                self.pool[n], self.pool[n + "_scale"] = c.to(torch.int8), d
                self.value[n] = (c.unflatten(-1, (-1, 32)) * d.double()[..., None]).flatten(-2)
        rand = lambda h: torch.randn((self.n_rows, h, dh), generator=g).to(device).to(self.dtype)  # noqa: E731
        self.q, self.gate = rand(hq), rand(hq)
        self.new_k, self.new_v = rand(hkv), rand(hkv)

    def ops(self):
        from speculative_decode_persistent_gb300 import ops
        p = self.pool
        return (ops.KVPool(p["k"], p["v"], p.get("k_scale"), p.get("v_scale")),
                ops.KVRows(self.start, self.kv_len, self.tables, self.n_rows, max([q for q, _ in self.seqs] + [0])))

    def gather(self, i, name):
        """(values [tokens][hkv][dh], exists [tokens]) of sequence i in double; tokens without a page are 0."""
        t = self.seqs[i][1]
        page = self.tables[i].long().repeat_interleave(16)[:t]
        ok = (page >= 0) & (page < self.n_pages)
        x = self.value[name][page.clamp(0, self.n_pages - 1), :, torch.arange(t, device=page.device) % 16]
        return torch.where(ok[:, None, None], x, 0.0), ok

    def attend_ref(self, window=0, sinks=0, gate=False, scale=None):
        """(out, bound) in double, [rows_used][hq][dh]; unseen values never enter."""
        scale = scale or self.dh ** -0.5
        outs, bounds, at = [], [], 0
        eps = torch.finfo(self.dtype).eps / 2
        for i, (n, T) in enumerate(self.seqs):
            if not n:
                continue
            k, ok = self.gather(i, "k")
            v, _ = self.gather(i, "v")
            q = self.q[at:at + n].double().view(n, self.hkv, self.hq // self.hkv, self.dh)
            gt = self.gate[at:at + n].double().view(n, self.hkv, self.hq // self.hkv, self.dh)
            at += n
            t = torch.arange(T, device=k.device)
            p = torch.arange(T - n, T, device=k.device)[:, None]
            see = (t <= p) & ok
            if window:
                see &= (p - t < window) | (t < sinks)
            see4 = see[:, None, None, :]
            s = torch.einsum("nhgd,thd->nhgt", q, torch.nan_to_num(k)) * scale
            bad = torch.einsum("nhgd,thd->nhgt", q, k) * scale  # nan / inf of seen tokens count
            s = torch.where(torch.isfinite(bad), s, bad)
            s = torch.where(see4, s, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(s - m)
            tot = w.sum(-1, keepdim=True)
            w = torch.where(tot > 0, w / tot, torch.where(torch.isnan(tot), tot, 0.0))
            fin = torch.where(torch.isfinite(v), v, 0.0)
            o = torch.einsum("nhgt,thd->nhgd", w, fin)
            a = torch.einsum("nhgt,thd->nhgd", torch.nan_to_num(w), fin.abs())
            # seen infinities and NaN of v: their sign, NaN where they disagree
            inf = lambda mask: torch.einsum("nt,thd->nhd", see.double(), mask.double())[:, :, None, :] > 0  # noqa: E731
            pi, ni, na = inf(v == math.inf), inf(v == -math.inf), inf(torch.isnan(v))
            o = torch.where(pi, o + math.inf, torch.where(ni, o - math.inf, o))  # a NaN stays one
            o = torch.where(na | (pi & ni), math.nan, o)
            # ---- the error that the roundings allow (u = 2^-11, half a binary16 step)
            u = 2.0 ** -11
            # scores: fp32 sums of dh exact products, each addition cut at 2^-23 of the
            # partial sum; a q8 key value is rounded to binary16 on top
            sa = torch.einsum("nhgd,thd->nhgt", q.abs(), torch.nan_to_num(k).abs()) * scale
            sa = torch.where(see4, sa, 0.0).amax(-1, keepdim=True)
            e = sa * (self.dh * 2.0 ** -23 + (u if self.kv == "q8" else 0.0)) + 2.0 ** -20 * (1 + m.abs())
            rel = torch.expm1(torch.nan_to_num(e).clamp_max(5.0))
            b = rel * (a + torch.nan_to_num(o, posinf=0, neginf=0).abs())
            # probabilities are rounded to binary16 (smallest step 2^-24, the largest is at
            # least 1 and the sum too), q8 values too, sums are fp32
            b = b + a * (u + (u if self.kv == "q8" else 0.0) + 2 * T * 2.0 ** -23) + T * 2.0 ** -25 * fin.abs().amax()
            if gate:
                sg = torch.sigmoid(gt)
                o, b = o * sg, b * sg + o.abs().nan_to_num(posinf=0) * 2.0 ** -20
            b = b + (o.abs().nan_to_num(posinf=0) + b) * eps + torch.finfo(self.dtype).smallest_normal * 2.0 ** -10
            outs.append(o.reshape(n, self.hq, self.dh))
            bounds.append(b.reshape(n, self.hq, self.dh))
        if not outs:
            z = torch.zeros((0, self.hq, self.dh), dtype=torch.double, device=self.q.device)
            return z, z
        return torch.cat(outs), torch.cat(bounds)


def assert_within(got, want, bound):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN elsewhere than the definition has them"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), "infinities differ"
    err = (got - want).abs()[fin]
    over = err - bound[fin]
    assert not over.numel() or float(over.max()) <= 0, (float(err.max()), float(over.max()), int((over > 0).sum()))
