"""Plain models of the attention layers' calls, for the tests: 64-bit arithmetic (where its inputs lie), sharing nothing with the
library, with bounds on what the calls' arithmetic may differ by."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24                                               # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of a type, relative
LEAST = -100                                                 # exponent of the smallest e4m3 scale


def attend(q, k, v, seen, scale, p_half):
    """(o, slack) of rows q [n][dk] over the first seen[i] (int) of k [m][dk], v [m][dv], in float64.

    Slack, with u the half step of fp32 and A_ij = scale sum_c |q_c k_c|: a score is a sum of d products in fp32, each
    addition off by at most 2 u of the sum of sizes (the matrix cores may cut where others round), and is multiplied by the
    scale and by log2(e) and has the maximum taken off: |ds| <= E_i = max_j (2 (d + 2) + 6) u A_ij + 4 u max |s|.  A power
    is then off by E + 2 u, the sum and the products over n keys by another 2 n u each, the quotient by 2 u; the
    probabilities are rounded by `p_half` before the product.  All of it is relative to sum_j p_ij |v_j|."""
    q, k, v = q.double(), k.double(), v.double()
    n, m, d = q.shape[0], k.shape[0], q.shape[1]
    if m == 0:
        return q.new_zeros(n, v.shape[1]), q.new_zeros(n, v.shape[1])
    there = torch.arange(m, device=q.device) < torch.as_tensor(seen, device=q.device)[:, None]
    s = (q @ k.T) * scale
    s = torch.where(there, s, -math.inf)
    p = torch.softmax(s, -1)
    p = torch.where(there, p, 0.0)  # (rows that see nothing)
    used = there.any(0)  # (what nobody sees may be anything)
    k, v, p, s, there = k[used], v[used], p[:, used], s[:, used], there[:, used]
    if torch.isfinite(v).all():
        o = p @ v
    else:  # (0 times what a row does not see could be NaN)
        o = torch.stack([(p[:, :, None] * torch.where(there[:, :, None], v[None, :, c:c + 1], 0.0)).sum(1)[:, 0] for c in range(v.shape[1])], 1)
    size = torch.where(there, (q.abs() @ k.abs().T) * abs(scale), 0.0)
    e = (2 * (d + 2) + 6) * U * size.amax(1) + 4 * U * torch.where(there, s.abs(), 0.0).amax(1) if there.shape[1] else q.new_zeros(n)
    va = torch.where(torch.isfinite(v), v, 0.0).abs()
    return o, (2 * (e + 2 * U) + p_half + 4 * m * U + 2 * U)[:, None] * (p @ va)


def close(got, ref, slack, what=""):
    """got is the rounding (of its type) of a value within slack of ref; NaN passes only where ref is not finite."""
    ref, slack = ref.to(got.device), slack.to(got.device)
    g, fine = got.double(), torch.isfinite(ref)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)}, not {tuple(ref.shape)}"
    assert bool((torch.isfinite(g) == fine).all()), f"{what}: {int((torch.isfinite(g) != fine).sum())} values finite, or not, by mistake"
    tol = slack + HALF[got.dtype] * (ref.abs() + slack) + 1e-37
    off = (g - ref).abs()
    bad = fine & ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off / tol)[fine].max()):.3g} of the bound"


def fwd(q, k, v, scale, lens_q, lens_k=None):
    """(o, slack) of packed prompts: q [n][Hq][dk], k [m][Hk][dk], v [m][Hk][dv]."""
    lens_k = lens_q if lens_k is None else lens_k
    G = q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64, device=q.device)
    slack = torch.zeros_like(o)
    p_half = HALF[torch.bfloat16] if q.dtype == torch.bfloat16 else 0.0
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        seen = (torch.arange(n, device=q.device) + m - n + 1).clamp(min=0)
        for h in range(q.shape[1]):
            o[a:a + n, h], slack[a:a + n, h] = attend(q[a:a + n, h], k[b:b + m, h // G], v[b:b + m, h // G], seen, scale, p_half)
        a, b = a + n, b + m
    return o, slack


def scale_of(amax):
    """The e4m3 scale for values up to amax, by its definition."""
    e = LEAST
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def e4m3(x):
    """x (float64, anything) as e4m3 stands for it: ties to even, steps of 2^-9 below 2^-6; not finite: NaN."""
    fine = torch.isfinite(x)
    y = torch.where(fine, x, 0.0)
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.where(fine, torch.round(y / step) * step, math.nan)


def turn(x, pos, freq, pairing):
    """(y, slack): x [n][H][d] in float64 with its first 2 len(freq) values turned by pos.

    Slack: two products and a sum of fp32, a cosine and a sine off by 4 u for the function, 7 u for the angle's rounding to
    fp32 after its reduction (an angle within pi: at most 2 pi u) and 8 u for the fp64 angle of far positions: under 32 u of
    |a| + |b|."""
    y = x.double().clone()
    size = torch.zeros_like(y)
    if freq is not None and len(freq):
        r = 2 * len(freq)
        f = torch.as_tensor(pos, dtype=torch.float64)[:, None] * freq.double().cpu()
        c, s = torch.cos(f)[:, None], torch.sin(f)[:, None]
        i = torch.arange(r // 2)
        a, b = (i, i + r // 2) if pairing == "halves" else (2 * i, 2 * i + 1)
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = ya.abs() + yb.abs()
    return y, 32 * U * size


class Pages:
    """A pool as lists of pages in float64: k [P][H][pt][dk], v, scales [P][2][H] (None: bf16)."""

    def __init__(self, layout, pool):
        k, v, s = layout.views(pool.cpu())
        self.layout, self.kv = layout, [k.double().clone(), v.double().clone()]
        self.scales = None if s is None else s.double().clone()

    def tokens(self, row, n):
        """The first n tokens on the pages of a row (a page out of range: None) as (keys, values, there)."""
        pt, P = self.layout.page_tokens, self.kv[0].shape[0]
        out, there = [], []
        for i, x in enumerate(self.kv):
            y = torch.zeros(max(n, 0), self.layout.H, x.shape[3], dtype=torch.float64)
            for j in range(-(-n // pt)):
                page = row[j] if j < len(row) else -1
                m = min(pt, n - j * pt)
                ok = 0 <= page < P
                if ok:
                    z = x[page, :, :m]
                    y[j * pt:j * pt + m] = (z if self.scales is None else z * self.scales[page, i][:, None, None]).transpose(0, 1)
                if i == 0:
                    there += [ok] * m
            out.append(y)
        return (*out, torch.tensor(there, dtype=torch.bool))

    def append(self, rows, before, k, v):
        """Each sequence's new keys and values (lists of [n][H][d] in float64) behind its `before` tokens."""
        pt, P = self.layout.page_tokens, self.kv[0].shape[0]
        touched = {}
        for b, row in enumerate(rows):
            for j in range(before[b] // pt, -(-(before[b] + k[b].shape[0]) // pt) if k[b].shape[0] else 0):
                page = row[j] if row is not None and j < len(row) else -1
                if 0 <= page < P:
                    touched.setdefault(page, []).append((b, j))
        for page, who in touched.items():
            if len(who) > 1:
                continue
            b, j = who[0]
            lo, hi = max(before[b], j * pt), min(before[b] + k[b].shape[0], (j + 1) * pt)
            for i, new in enumerate((k[b], v[b])):
                x = new[lo - before[b]:hi - before[b]].transpose(0, 1)
                held = self.kv[i][page]
                if self.scales is None:
                    held[:, lo - j * pt:hi - j * pt] = x
                    continue
                for h in range(x.shape[0]):
                    fine = x[h][torch.isfinite(x[h])]
                    s = scale_of(float(fine.abs().max()) if fine.numel() else 0.0)
                    if lo > j * pt:
                        was = float(self.scales[page, i, h])
                        s = max(s, was)
                        held[h, :lo - j * pt] = e4m3(held[h, :lo - j * pt] * (was / s))
                    held[h, lo - j * pt:hi - j * pt] = e4m3(x[h] / s)
                    self.scales[page, i, h] = s
