"""The operators of the attention layers that stand between the recurrent ones: what one pass of each is, on which
inputs.

* ``prompt``: attention over whole prompts, causal, grouped heads, packed sequences of different lengths, with or
  without a prefix whose keys are there already (``kda_attn_fwd``);
* ``append``: new tokens' keys and values turned by position and put on the pages of a cache in bf16 or e4m3
  (``kda_kv_append``), the queries turned beside them;
* ``read``: cached tokens back as dense rows (``kda_kv_read``);
* ``decode``: one token, or a few drafted ones, of each sequence against its cached tokens (``kda_attn_decode``).

A page holds ``pt`` tokens: the keys [Hk][pt][dk], the values [Hk][pt][dv] and, in e4m3, a scale for each head's
keys and values on the page: the smallest power of two, at least 2^-100, that brings the largest finite of them to 448 or below.

``own`` false: the plain form of the operator in elementary torch operations.  True: the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_BF, _F, _E = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_DT = {"bf16": _BF, "f32": _F, "e4m3": _E}
_LEAST = -100  # exponent of the smallest scale


# ---- the cases ------------------------------------------------------------------------------------


def listed():
    return [
        # a chat's first line on a small layer: latency
        dict(name="prompt short", kind="prompt", N=1, total=77, prefix=0, Hq=8, Hk=2, dk=64, dv=64, dtype="bf16", fused=True),
        # a batch of prompts of very different lengths, packed, 32 + 8 heads of 128
        dict(name="prompt packed", kind="prompt", N=16, total=24961, prefix=0, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16", fused=True),
        # one long document
        dict(name="prompt 16K", kind="prompt", N=1, total=16384, prefix=0, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16", fused=False),
        # the next turns of 3 chats at full precision, behind prefixes that are cached
        dict(name="prompt turns f32", kind="prompt", N=3, total=391, prefix=1500, Hq=8, Hk=4, dk=64, dv=128, dtype="f32", fused=False),
        # one chat's next token in fp32 on a small layer: latency
        dict(name="append token", kind="append", N=1, pad=0, total=1, before=901, Hq=8, Hk=2, dk=64, dv=64, dtype="f32", cache="bf16",
             pt=16, rot=64, pairing="pairs"),
        # a captured batch of 256 rows, 6 of them padding, one token each into 8-bit pages
        dict(name="append 256", kind="append", N=256, pad=6, total=256, before=2000, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16",
             cache="e4m3", pt=64, rot=128, pairing="halves"),
        # 16 prompts of 64K tokens in all, some behind a cached prefix that ends inside a page
        dict(name="append prompts 64K", kind="append", N=16, pad=0, total=65536, before=100, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16",
             cache="e4m3", pt=64, rot=64, pairing="halves"),
        # one chat's short history on bf16 pages, back for its next turn
        dict(name="read one", kind="read", N=1, total=517, Hk=4, dk=64, dv=128, cache="bf16", out="bf16", pt=32),
        # the prefixes of 8 chats, back from 8-bit pages
        dict(name="read 8 prefixes", kind="read", N=8, total=70001, Hk=8, dk=128, dv=128, cache="e4m3", out="bf16", pt=64),
        # one chat's next token
        dict(name="decode one", kind="decode", B=1, pad=0, K=1, lo=903, hi=903, Hq=8, Hk=2, dk=64, dv=64, dtype="bf16", cache="bf16", pt=16),
        # a batch of 256 rows, 6 of them padding, 300 to 9,000 tokens on 8-bit pages
        dict(name="decode 256", kind="decode", B=256, pad=6, K=1, lo=300, hi=9000, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16",
             cache="e4m3", pt=64),
        # 4 drafted tokens of one chat with a 1M-token context on 8-bit pages
        dict(name="decode 1M drafts", kind="decode", B=1, pad=0, K=4, lo=1000003, hi=1000003, Hq=32, Hk=8, dk=128, dv=128, dtype="bf16",
             cache="e4m3", pt=128),
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "append", "append", "read", "decode", "decode"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 5, 8])
    if kind == "prompt":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 64), (128, 64), (32, 16)])
        N = _log(rng, 1, 24)
        total = max(N, _log(rng, 1, 12000 if dtype == "bf16" else 2000))
        return dict(kind=kind, N=N, total=total, prefix=rng.choice([0, 0, _log(rng, 1, 2000)]), Hq=Hq, Hk=Hk, dk=dk, dv=dv, dtype=dtype,
                    fused=rng.random() < 0.5)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    cache, pt = rng.choice(["e4m3", "e4m3", "bf16"]), rng.choice([16, 32, 64, 64, 128])
    if kind == "append":
        N = _log(rng, 1, 256)
        total = N if rng.random() < 0.5 else max(N, _log(rng, 1, 40000))
        return dict(kind=kind, N=N, pad=rng.randint(0, N - 1) // 8, total=total, before=_log(rng, 1, 3000), Hq=Hq, Hk=Hk, dk=dk, dv=dv,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), cache=cache, pt=pt, rot=rng.choice([0, dk, 16, 32]),
                    pairing=rng.choice(["halves", "pairs"]))
    if kind == "read":
        N = _log(rng, 1, 64)
        return dict(kind=kind, N=N, total=max(N, _log(rng, 1, 60000)), Hk=Hk, dk=dk, dv=dv, cache=cache, out=rng.choice(["bf16", "bf16", "f32"]),
                    pt=pt)
    B, K = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 5])
    hi = _log(rng, K, max(K, min(200000, 600000 // B)))
    return dict(kind=kind, B=B, pad=rng.randint(0, B - 1) // 8, K=K, lo=rng.randint(K, hi), hi=hi, Hq=Hq, Hk=Hk, dk=dk, dv=dv,
                dtype=rng.choice(["bf16", "bf16", "f32"]), cache=cache, pt=pt)


# ---- inputs ---------------------------------------------------------------------------------------


def _split(total, N):
    """Lengths of N sequences that make up `total`, each at least 1 where that goes, from short to twenty times as long."""
    w = [1 + (i * 7919 + 3) % 20 for i in range(N)]
    lens = [max(1, total * x // sum(w)) for x in w]
    lens[-1] += total - sum(lens)
    while lens[-1] < 1:  # (few tokens for many sequences)
        i = max(range(N), key=lambda j: lens[j])
        lens[i], lens[-1] = lens[i] - 1, lens[-1] + 1
    return lens


def _spread(lo, hi, N):
    """N lengths between lo and hi, hi among them."""
    return [hi if b == N // 2 else lo + (b * 40503 % 997) * (hi - lo) // 996 for b in range(N)]


def _prefixes(c):
    return [0 if not c["prefix"] else c["prefix"] // 2 + (b * 379) % (c["prefix"] // 2 + 1) for b in range(c["N"])]


def _before(c):
    """Tokens that each sequence of an append has on its pages: none, some inside a page, whole pages."""
    return [c["before"]] if c["N"] == 1 else [(b * 53 % 7) * c["before"] // 6 // (c["pt"] if b % 5 == 0 else 1) * (c["pt"] if b % 5 == 0 else 1)
                                              for b in range(c["N"])]


def _ints(x, dev):
    return torch.as_tensor(x, dtype=torch.int32).to(dev)


def _cu(lens, dev):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)], dev)


def _keys(g, dev, *shape):
    """Values like a layer's keys: some channels much larger than the others."""
    x = torch.randn(*shape, generator=g, device=dev)
    x[..., ::16] *= 4.0
    return x


def _scales(amax):
    """The scale for values up to amax."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e - 9 + (m > 0.875).int(), _LEAST).clamp(min=_LEAST))


def _views(c, pool):
    """The pool's keys [P][Hk][pt][dk], values [P][Hk][pt][dv] and scales [P][2][Hk] (None in bf16)."""
    P, Hk, pt, dk, dv = pool.shape[0], c["Hk"], c["pt"], c["dk"], c["dv"]
    e = 1 if c["cache"] == "e4m3" else 2
    a, b = Hk * pt * dk * e, Hk * pt * (dk + dv) * e
    keys = pool[:, :a].view(_DT[c["cache"]]).unflatten(1, (Hk, pt, dk))
    values = pool[:, a:b].view(_DT[c["cache"]]).unflatten(1, (Hk, pt, dv))
    return keys, values, pool[:, b:b + 8 * Hk].view(_F).unflatten(1, (2, Hk)) if e == 1 else None


def _pool(c, need, g, h, dev):
    """Pages of cached tokens in random order, a table whose rows hold need[b] of them, and a few rows and pages of others."""
    N = len(need)
    P = sum(need) + 5
    Hk, pt, dk, dv = c["Hk"], c["pt"], c["dk"], c["dv"]
    size = Hk * pt * (dk + dv) * 2 if c["cache"] == "bf16" else Hk * pt * (dk + dv) + (8 * Hk + 15) // 16 * 16
    pool = torch.zeros(P, size, dtype=torch.uint8, device=dev)
    keys, values, scales = _views(c, pool)
    for i, (to, d) in enumerate(((keys, dk), (values, dv))):
        for p in range(0, P, 4096):
            x = _keys(g, dev, min(4096, P - p), Hk, pt, d) if i == 0 else torch.randn(min(4096, P - p), Hk, pt, d, generator=g, device=dev)
            if scales is not None:
                s = _scales(x.abs().amax((2, 3)))
                scales[p:p + 4096, i] = s
                x = x / s[:, :, None, None]
            to[p:p + 4096] = x.to(to.dtype)
    order = torch.randperm(P, generator=h).tolist()
    table = torch.full((N + 3, max(max(need), 1)), -1, dtype=torch.int32)
    rows = torch.randperm(N + 3, generator=h)[:N]
    for b, r in enumerate(rows.tolist()):
        table[r, :need[b]] = torch.tensor(order[sum(need[:b]):sum(need[:b + 1])], dtype=torch.int32)
    if c.get("pad"):
        rows[N - c["pad"]:] = -1
    return dict(pool=pool, table=table.to(dev), rows=_ints(rows, dev))


def _layout(c):
    import gated_delta_rule_07_amd as kda
    return kda.KVLayout(_DT[c["cache"]], c["pt"], c["Hk"], c["dk"], c["dv"])


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = dict(c=c)
    Hk, dk, dv = c["Hk"], c["dk"], c["dv"]
    if c["kind"] == "prompt":
        dt, n = _DT[c["dtype"]], c["total"]
        lens, pre = _split(n, c["N"]), _prefixes(c)
        m = n + sum(pre)
        if c["fused"] and dk == dv and m == n:  # rows of a fused projection
            row = torch.randn(n, c["Hq"] + 2 * Hk, dk, generator=g, device=dev).to(dt)
            s["q"], s["k"], s["v"] = row[:, :c["Hq"]], row[:, c["Hq"]:c["Hq"] + Hk], row[:, c["Hq"] + Hk:]
        else:
            s["q"] = torch.randn(n, c["Hq"], dk, generator=g, device=dev).to(dt)
            s["k"], s["v"] = _keys(g, dev, m, Hk, dk).to(dt), torch.randn(m, Hk, dv, generator=g, device=dev).to(dt)
        s["cu"], s["cu_k"] = _cu(lens, dev), _cu([a + b for a, b in zip(lens, pre)], dev) if sum(pre) else None
        s["lens"], s["pre"] = lens, pre  # (a server knows them on the host too)
        s["o"] = torch.zeros(n, c["Hq"], dv, dtype=dt, device=dev)
        return s
    if c["kind"] == "append":
        dt, n = _DT[c["dtype"]], c["total"]
        lens, before = _split(n, c["N"]), _before(c)
        s.update(_pool(c, [-(-(a + b) // c["pt"]) for a, b in zip(lens, before)], g, h, dev))
        s["q"] = torch.randn(n, c["Hq"], dk, generator=g, device=dev).to(dt)
        s["k"], s["v"] = _keys(g, dev, n, Hk, dk).to(dt), torch.randn(n, Hk, dv, generator=g, device=dev).to(dt)
        s["before"], s["cu"] = _ints(before, dev), None if n == c["N"] else _cu(lens, dev)
        s["freq"] = (10000.0 ** (-torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) / max(1, c["rot"] // 2))).float() if c["rot"] else None
        s["qo"] = torch.zeros_like(s["q"])
    elif c["kind"] == "read":
        lens = _split(c["total"], c["N"])
        s["starts"] = [b * 31 % 200 if b % 3 == 1 else 0 for b in range(c["N"])]  # (some from inside a page on)
        s.update(_pool(c, [-(-(a + b) // c["pt"]) for a, b in zip(lens, s["starts"])], g, h, dev))
        s["starts"], s["cu"] = _ints(s["starts"], dev), _cu(lens, dev)
        s["ko"], s["vo"] = (torch.zeros(c["total"], Hk, d, dtype=_DT[c["out"]], device=dev) for d in (dk, dv))
    else:
        lens = _spread(c["lo"], c["hi"], c["B"])
        s.update(_pool(c, [-(-x // c["pt"]) for x in lens], g, h, dev))
        s["q"] = torch.randn(c["B"], c["K"], c["Hq"], dk, generator=g, device=dev).to(_DT[c["dtype"]])
        s["lens"] = _ints(lens, dev)
        s["o"] = torch.zeros(c["B"], c["K"], c["Hq"], dv, dtype=_DT[c["dtype"]], device=dev)
    s["scale"] = dk ** -0.5
    return s


# ---- one pass -------------------------------------------------------------------------------------


def run(state):
    return {"prompt": _prompt, "append": _append, "read": _read, "decode": _decode}[state["c"]["kind"]](state)


def _attend(q, k, v, first, scale):
    """q [Hk][G][n][dk] against k [Hk][m][dk], v [Hk][m][dv], in fp32: query i attends to keys 0 .. first + i."""
    score = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, q.shape[1:3]) * scale
    i, j = torch.arange(q.shape[2], device=q.device), torch.arange(k.shape[1], device=q.device)
    score.masked_fill_(j > i[:, None] + first, -math.inf)
    score = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    return torch.matmul(score.flatten(1, 2), v).unflatten(1, q.shape[1:3]) / score.sum(-1, keepdim=True)


def _prompt(s):
    c = s["c"]
    if own:
        import gated_delta_rule_07_amd as kda
        return kda.kda_attn_fwd(s["q"], s["k"], s["v"], scale=c["dk"] ** -0.5, cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"], o=s["o"])
    G, at, ak = c["Hq"] // c["Hk"], 0, 0
    for n, pre in zip(s["lens"], s["pre"]):  # a sequence's scores take the square of its length: one after another, in slices
        k, v = (s[x][ak:ak + pre + n].float().transpose(0, 1) for x in ("k", "v"))
        step = max(1, min(n, (1 << 30) // (c["Hq"] * (n + pre))))
        for i in range(0, n, step):
            q = s["q"][at + i:at + min(n, i + step)].float().unflatten(1, (c["Hk"], G)).permute(1, 2, 0, 3)
            last = pre + min(n, i + step)
            o = _attend(q, k[:, :last], v[:, :last], pre + i, c["dk"] ** -0.5)
            s["o"][at + i:at + min(n, i + step)] = o.permute(2, 0, 1, 3).flatten(1, 2).to(s["o"].dtype)
        at, ak = at + n, ak + pre + n
    return s["o"]


def _turn(x, pos, s):
    """x [n][H][d] in fp32, its first rot values turned by position."""
    c, r = s["c"], s["c"]["rot"]
    if not r:
        return x
    angle = pos.double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if c["pairing"] == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _places(s, n):
    """Of each of n tokens: its sequence, its position, its page and whether that is one."""
    c, dev = s["c"], s["table"].device
    first = s["before"] if "before" in s else s["starts"]
    at = torch.arange(n, device=dev)
    b = at if s["cu"] is None else torch.searchsorted(s["cu"][1:], at, right=True)
    pos = first[b] + (0 if s["cu"] is None else at - s["cu"][b])
    row = s["rows"][b]
    page = torch.where(row >= 0, s["table"][row.clamp(min=0), pos // c["pt"]], -1)
    return b, pos, page, page >= 0


def _append(s):
    c = s["c"]
    if own:
        import gated_delta_rule_07_amd as kda
        kda.kda_kv_append(s["k"], s["v"], s["pool"], _layout(c), s["table"], s["before"], rows=s["rows"], cu_seqlens=s["cu"], q=s["q"],
                          inv_freq=s["freq"], pairing=c["pairing"], q_out=s["qo"])
        return [s["qo"], *(x for x in _views(c, s["pool"]) if x is not None)]
    b, pos, page, there = _places(s, c["total"])
    s["qo"].copy_(_turn(s["q"].float(), pos, s))
    keys, values, scales = _views(c, s["pool"])
    page, slot = page[there].long(), (pos % c["pt"])[there]
    new = (_turn(s["k"].float(), pos, s)[there], s["v"].float()[there])
    if scales is not None:
        # a sequence's first page may hold tokens: their scale stays where it is enough, and they are rounded to the new one where not
        held = (s["rows"] >= 0) & (s["before"] % c["pt"] > 0)
        at = s["table"][s["rows"].clamp(min=0), (s["before"] // c["pt"]).clamp(max=s["table"].shape[1] - 1)]
        old, count = at[held].long(), (s["before"] % c["pt"])[held]
    for i, (to, x) in enumerate(zip((keys, values), new)):
        if scales is not None:
            was = scales[old, i]
            amax = torch.zeros(len(scales), c["Hk"], device=x.device).index_reduce_(0, page, x.abs().amax(-1), "amax")
            now = _scales(amax)
            now[old] = torch.maximum(now[old], was)
            again = (to[old].float() * (was / now[old])[..., None, None]).to(_E)
            mine = torch.arange(c["pt"], device=x.device) < count[:, None]
            to[old] = torch.where(mine[:, None, :, None], again.view(torch.uint8), to[old].view(torch.uint8)).view(_E)
            scales[page, i] = now[page]
            x = x / now[page][..., None]
        to[page, :, slot] = x.to(to.dtype)
    return [s["qo"], *(x for x in (keys, values, scales) if x is not None)]


def _read(s):
    c = s["c"]
    if own:
        import gated_delta_rule_07_amd as kda
        return list(kda.kda_kv_read(s["pool"], _layout(c), s["table"], s["cu"], c["total"], rows=s["rows"], starts=s["starts"], k_out=s["ko"],
                                    v_out=s["vo"]))
    _, pos, page, _ = _places(s, c["total"])
    keys, values, scales = _views(c, s["pool"])
    for i, (x, to) in enumerate(((keys, s["ko"]), (values, s["vo"]))):
        y = x[page.long(), :, pos % c["pt"]].float()
        to.copy_(y if scales is None else y * scales[page.long(), i][..., None])
    return [s["ko"], s["vo"]]


def _cached(c, pool, pages):
    """Keys and values [..][tokens][Hk][d] of the pages in fp32; -1: zeros."""
    keys, values, scales = _views(c, pool)
    for i, x in enumerate((keys, values)):
        y = x[pages.clamp(min=0).long()].float()
        if scales is not None:
            y *= scales[pages.clamp(min=0).long(), i][..., None, None]
        yield (y * (pages >= 0)[..., None, None, None]).transpose(-2, -3).flatten(-4, -3)


def _decode(s):
    c = s["c"]
    if own:
        import gated_delta_rule_07_amd as kda
        return kda.kda_attn_decode(s["q"], s["pool"], _layout(c), s["table"], s["lens"], rows=s["rows"], scale=s["scale"], o=s["o"])
    B, K, Hk, G = c["B"] - c["pad"], c["K"], c["Hk"], c["Hq"] // c["Hk"]  # the padding of a batch stands at its end
    part = max(1, min(B, (24 << 30) // (s["table"].shape[1] * c["pt"] * Hk * (c["dk"] + c["dv"]) * 4)))
    for b in range(0, B, part):  # (as many sequences at once as have room for their keys and values in fp32)
        e = min(B, b + part)
        k, v = _cached(c, s["pool"], s["table"][s["rows"][b:e]])
        q = s["q"][b:e].float().unflatten(2, (Hk, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
        score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
        seen = s["lens"][b:e, None] - K + 1 + torch.arange(K, device=q.device)
        hidden = torch.arange(k.shape[1], device=q.device) >= seen[..., None]
        score.masked_fill_(hidden.repeat_interleave(G, 1)[:, None], -math.inf)
        score = torch.exp(score - score.amax(-1, keepdim=True))
        o = torch.matmul(score, v.transpose(1, 2)) / score.sum(-1, keepdim=True)
        s["o"][b:e] = o.unflatten(2, (K, G)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["o"].dtype)
    return s["o"]


# ---- what a pass cannot do without ----------------------------------------------------------------


def work(case):
    c = case
    Hk, dk, dv = c["Hk"], c["dk"], c["dv"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["kind"] == "prompt":
        lens, pre = _split(c["total"], c["N"]), _prefixes(c)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, pre))
        values = c["total"] * c["Hq"] * (dk + dv) + (c["total"] + sum(pre)) * Hk * (dk + dv)
        return dict(bytes=values * size[c["dtype"]] + 8 * c["N"], flops=2 * pairs * c["Hq"] * (dk + dv))
    if c["kind"] == "append":
        n = c["total"] - sum(_split(c["total"], c["N"])[c["N"] - c["pad"]:])
        row = Hk * (dk + dv)
        return dict(bytes=c["total"] * 2 * c["Hq"] * dk * size[c["dtype"]] + n * row * (size[c["dtype"]] + size[c["cache"]]) + 12 * c["N"],
                    flops=3 * c["total"] * (c["Hq"] + Hk) * c["rot"] + n * row)
    if c["kind"] == "read":
        return dict(bytes=c["total"] * Hk * (dk + dv) * (size[c["cache"]] + size[c["out"]]) + 12 * c["N"], flops=0)
    lens = _spread(c["lo"], c["hi"], c["B"])[:c["B"] - c["pad"]]
    pairs = sum(c["K"] * n - c["K"] * (c["K"] - 1) // 2 for n in lens)
    return dict(bytes=sum(lens) * Hk * (dk + dv) * size[c["cache"]] + (len(lens) * c["K"]) * c["Hq"] * (dk + dv) * size[c["dtype"]]
                + 4 * sum(-(-n // c["pt"]) for n in lens), flops=2 * pairs * c["Hq"] * (dk + dv))


# ---- the definitions, in 64 bits ------------------------------------------------------------------


def _round_e4m3(x):
    """x in float64 (at most 448) rounded to e4m3, ties to even: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _scale64(amax):
    e = _LEAST if not amax > 0 else max(_LEAST, math.ceil(math.log2(amax)) - 10)
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _softmax_rows(q, k, v, seen, scale):
    """Rows q [n][dk] over the first seen[i] of k [m][dk], v [m][dv], in float64."""
    t = (q @ k.T) * scale
    t = torch.where(torch.arange(len(k), device=q.device) < seen[:, None], t, -math.inf)
    return torch.softmax(t, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, torch.device("cuda")
    G = c.get("Hq", 0) // c["Hk"]
    if c["kind"] == "prompt":
        o = torch.zeros_like(s["o"], dtype=torch.float64)
        at = ak = 0
        for n, pre in zip(s["lens"], s["pre"]):
            for h in range(c["Hq"]):
                k, v = s["k"][ak:ak + n + pre, h // G].double(), s["v"][ak:ak + n + pre, h // G].double()
                for i in range(0, n, 4096):
                    rows = slice(at + i, at + min(n, i + 4096))
                    seen = pre + 1 + torch.arange(i, min(n, i + 4096), device=dev)
                    o[rows, h] = _softmax_rows(s["q"][rows, h].double(), k, v, seen, c["dk"] ** -0.5)
            at, ak = at + n, ak + n + pre
        return o
    keys, values, scales = _views(c, s["pool"])
    if c["kind"] == "read":
        table, rows, out = s["table"].tolist(), s["rows"].tolist(), []
        cu, starts = s["cu"].tolist(), s["starts"].tolist()
        for i, (x, to) in enumerate(((keys, s["ko"]), (values, s["vo"]))):
            y = torch.zeros_like(to, dtype=torch.float64)
            for b in range(c["N"]):
                pages = torch.tensor(table[rows[b]], device=dev).clamp(min=0)
                z = x[pages].double() if scales is None else x[pages].double() * scales[pages, i].double()[..., None, None]
                y[cu[b]:cu[b + 1]] = z.transpose(1, 2).flatten(0, 1)[starts[b]:starts[b] + cu[b + 1] - cu[b]]
            out.append(y)
        return out
    if c["kind"] == "decode":
        o = s["o"].double()
        for b, n in enumerate(s["lens"].tolist()[:c["B"] - c["pad"]]):
            pages = s["table"][int(s["rows"][b])].long()[:-(-n // c["pt"])]
            for h in range(c["Hk"]):
                k, v = (x[pages, h].double() * (1.0 if scales is None else scales[pages, i, h].double()[:, None, None])
                        for i, x in enumerate((keys, values)))
                q = s["q"][b, :, h * G:(h + 1) * G].double().flatten(0, 1)
                seen = (n - c["K"] + 1 + torch.arange(c["K"], device=dev)).repeat_interleave(G)
                o[b, :, h * G:(h + 1) * G] = _softmax_rows(q, k.flatten(0, 1), v.flatten(0, 1), seen, s["scale"]).unflatten(0, (c["K"], G))
        return o
    # append: each pair of values as a complex number, turned; pages one after another
    lens, before, r = _split(c["total"], c["N"]), _before(c), c["rot"]
    pos = torch.cat([torch.arange(a, a + n, device=dev) for a, n in zip(before, lens)]).double()
    turned = []
    for x in (s["q"].double(), s["k"].double()):
        if r:
            i = torch.arange(r // 2, device=dev)
            a, b = (i, i + r // 2) if c["pairing"] == "halves" else (2 * i, 2 * i + 1)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), pos[:, None] * s["freq"].double()[None])
            pair = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            x[..., a], x[..., b] = pair.real, pair.imag
        turned.append(x)
    table, rows, at = s["table"].tolist(), s["rows"].tolist(), 0
    held = [keys.double(), values.double()]
    scale = None if scales is None else scales.double()
    for b, n in enumerate(lens):
        done = 0
        while done < n:
            slot = (before[b] + done) % c["pt"]
            m = min(n - done, c["pt"] - slot)
            page = table[rows[b]][(before[b] + done) // c["pt"]] if rows[b] >= 0 else -1
            if page >= 0:
                for i, x in enumerate((turned[1], s["v"].double())):
                    x = x[at + done:at + done + m].transpose(0, 1)
                    if scale is not None:
                        now = torch.tensor([_scale64(y) for y in x.abs().amax((1, 2)).tolist()], dtype=torch.float64, device=dev)
                        if slot:
                            now = torch.maximum(now, scale[page, i])
                            held[i][page, :, :slot] = _round_e4m3(held[i][page, :, :slot] * (scale[page, i] / now)[:, None, None])
                        scale[page, i] = now
                        x = _round_e4m3(x / now[:, None, None])
                    held[i][page, :, slot:slot + m] = x
            done += m
        at += n
    return [turned[0], *held] + ([] if scale is None else [scale])
