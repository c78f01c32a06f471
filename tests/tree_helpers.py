"""Cases and 64-bit references for the operators on trees of drafts: written
from the definitions, row by row, in double, sharing no code with the package.
Tolerances count roundings (derived where they stand), not measured values."""
import math

import torch

from ops_helpers import Case

U16 = 2.0 ** -11  # half a binary16 step, relative


def lineage(parents):
    """Each node's ancestors, from the root on, and itself; of one tree, by the documented rule."""
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if 0 <= p < j else []) + [j])
    return out


def random_parents(seqs, seed=0, kind="random"):
    g = torch.Generator().manual_seed(seed)
    out = []
    for q, _ in seqs:
        for j in range(q):
            if kind == "chain":
                out.append(j - 1)
            elif kind == "star":
                out.append(0 if j else -1)
            else:
                out.append(-1 if j == 0 else int(torch.randint(-1 if kind == "forest" else 0, j, (1,), generator=g)))
    return out


class TreeCase(Case):
    """A Case whose new rows are trees."""

    def __init__(self, seqs, *args, kind="random", parents=None, **kw):
        super().__init__(seqs, *args, **kw)
        device = self.q.device
        self.parent_list = list(parents) if parents is not None else random_parents(seqs, kw.get("seed", 0) + 99, kind)
        pad = [0] * (self.n_rows - self.rows_used)
        self.parents = torch.tensor(self.parent_list + pad, dtype=torch.int32, device=device)
        self.lines, at = [], 0
        for q, _ in seqs:
            self.lines.append(lineage(self.parent_list[at:at + q]))
            at += q

    def positions(self, i):
        q, T = self.seqs[i]
        return [T - q + len(line) - 1 for line in self.lines[i]]

    def sees(self, i, window, sinks):
        """[nodes][tokens] of sequence i."""
        q, T = self.seqs[i]
        base, see = T - q, torch.zeros(q, T, dtype=torch.bool)
        for j, line in enumerate(self.lines[i]):
            if base + j < 0:
                continue  # a row without a slot sees nothing
            pos = base + len(line) - 1
            t = torch.arange(max(base, 0))
            see[j, :max(base, 0)] = (pos - t < window) | (t < sinks) if window else True
            for depth, n in enumerate(line):
                if base + n >= 0:
                    see[j, base + n] = not window or pos - (base + depth) < window or base + depth < sinks
        return see.to(self.q.device)

    def tree_ref(self, window=0, sinks=0, gate=False, scale=None):
        """(out, bound) in double, [rows_used][hq][dh]; unseen values never enter."""
        scale = scale or self.dh ** -0.5
        outs, bounds, at = [], [], 0
        eps = torch.finfo(self.dtype).eps / 2
        for i, (n, T) in enumerate(self.seqs):
            if not n:
                continue
            k, ok = self.gather(i, "k")
            v, _ = self.gather(i, "v")
            shape = (n, self.hkv, self.hq // self.hkv, self.dh)
            q, gt = self.q[at:at + n].double().view(shape), self.gate[at:at + n].double().view(shape)
            at += n
            see = self.sees(i, window, sinks) & ok
            see4 = see[:, None, None, :]
            s = torch.einsum("nhgd,thd->nhgt", q, torch.nan_to_num(k)) * scale
            s = torch.where(see4, s, -math.inf)
            m = s.amax(-1, keepdim=True) if T else torch.full(shape[:3] + (1,), -math.inf, dtype=torch.double, device=k.device)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(s - m)
            tot = w.sum(-1, keepdim=True)
            w = torch.where(tot > 0, w / tot, 0.0)
            fin = torch.where(torch.isfinite(v), v, 0.0)
            o = torch.einsum("nhgt,thd->nhgd", w, fin)
            a = torch.einsum("nhgt,thd->nhgd", w, fin.abs())
            hits = lambda mask: torch.einsum("nt,thd->nhd", see.double(), mask.double())[:, :, None, :] > 0  # noqa: E731
            pi, ni, na = hits(v == math.inf), hits(v == -math.inf), hits(torch.isnan(v))
            o = torch.where(pi, o + math.inf, torch.where(ni, o - math.inf, o))
            o = torch.where(na | (pi & ni), math.nan, o)
            # what the documented roundings allow: scores are fp32 sums of dh products (each addition cut at 2^-23 of
            # the partial sum), q8 values are rounded to binary16; probabilities too (the smallest kept is 2^-25 of the
            # largest); sums are fp32; a sigmoid is off by 2^-20; one rounding to the output's type
            q8 = U16 if self.kv == "q8" else 0.0
            sa = torch.einsum("nhgd,thd->nhgt", q.abs(), torch.nan_to_num(k).abs()) * scale
            sa = torch.where(see4, sa, 0.0).amax(-1, keepdim=True) if T else m
            e = sa * (self.dh * 2.0 ** -23 + q8) + 2.0 ** -20 * (1 + m.abs())
            b = torch.expm1(e.clamp_max(5.0)) * (a + torch.nan_to_num(o, posinf=0, neginf=0).abs())
            b = b + a * (U16 + q8 + 2 * T * 2.0 ** -23)
            if T:
                b = b + T * 2.0 ** -25 * fin.abs().amax()
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


def turned(x, pos, rot, freq, gain, eps):
    """(values, bound on an fp32 evaluation's error) of x [rows][heads][dh] normalised and rotated, in double.

    freq [rot / 2]: radians a position. The bound, with u = 2^-24 an fp32 rounding: the norm's factor carries its sum
    (pairwise at worst dh u), one division, an addition, a reciprocal root within 2 ulp (4 u) and a product, so
    (dh + 8) u; gain and product 2 u; the angle is off by 2^-25 of a turn (a 32-bit signed fraction rounded to 24
    bits: 2^-24 half turns) or 2^-23 radians, sine and cosine by 2 ulp more (4 u); the turn takes two products and a
    sum (3 u) of values of at most |x_i| + |x_j|."""
    u = 2.0 ** -24
    x = x.double()
    rel = 0.0
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
        rel = (x.shape[-1] + 10) * u
    a = torch.as_tensor(pos, dtype=torch.double, device=x.device)[:, None] * freq
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    # the definition's own angle, pos x freq in double, is off by an ulp of it: its turns too, where pos is large
    slack = (a.abs() * 2.0 ** -51)[:, None]
    h = rot // 2
    lo, hi, rest = x[..., :h], x[..., h:rot], x[..., rot:]
    size = lo.abs() + hi.abs()
    out = torch.cat([lo * c - hi * s, hi * c + lo * s, rest], -1)
    b = size * (rel + 2.0 ** -23 * math.pi + 8 * u + slack)
    return out, torch.cat([b, b, rest.abs() * (rel + u)], -1)


def walk(parents, tokens, logits):
    """(path, emitted) of one tree by the definition; logits a list of rows (lists of floats)."""
    path, out = [0], []
    while True:
        row = logits[path[-1]]
        g = -1 if any(math.isnan(x) for x in row) else max(range(len(row)), key=lambda i: (row[i], -i))
        out.append(g)
        nxt = [c for c in range(1, len(parents)) if parents[c] == path[-1] and c > path[-1] and g >= 0 and tokens[c] == g]
        if not nxt:
            return path, out
        path.append(nxt[0])
