"""The serving operators around the recurrent state: what one pass of each is, on which inputs.

Four groups, in the order in which a serving step uses them:

* ``heads``: queries and keys normalised for each head and rotated by position (``kda_qk_norm``), what a
  layer does to its projections before the recurrence reads them;
* ``fork`` / ``compact``: the cache of state pages (``kda_cache_fork``, ``kda_cache_copy``,
  ``kda_cache_free``, ``kda_cache_compact``);
* ``decode``: one token for each sequence on the pages of that cache (``kda_decode_step_paged``);
* ``verify`` / ``step``: a tree of drafted tokens over the cached states (``kda_tree_verify``), and the
  accepted path written back (``kda_tree_commit``).

``own`` false: the plain form of the operator in elementary torch operations.  True: the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_BF, _F = torch.bfloat16, torch.float32
_DT = {"bf16": _BF, "f32": _F}


# ---- the cases ------------------------------------------------------------------------------------


def listed():
    return [
        # a chat's next token on a small layer, its projections still in one fused row: latency
        dict(name="heads token", kind="heads", n=1, hq=8, hk=8, d=128, dtype="bf16", norm="l2", rot=0, pairing="halves",
             fused=True, weights=False, start=0),
        # the 64K prompt that the prefill benchmark runs, 32 heads of 128
        dict(name="heads prompt 64K", kind="heads", n=65536, hq=32, hk=32, d=128, dtype="bf16", norm="l2", rot=0,
             pairing="halves", fused=False, weights=False, start=0),
        # an attention layer beside the recurrent ones: grouped heads, learned weights, half of each head
        # rotated, a ragged chunk far into a 1M-token context
        dict(name="heads rotated chunk", kind="heads", n=4099, hq=32, hk=4, d=64, dtype="f32", norm="rms", rot=32,
             pairing="halves", fused=True, weights=True, start=900001),
        # one chat answered twice: its state (8 heads of 128 in 4 layers) copied to a second page
        dict(name="fork one", kind="fork", layers=4, H=8, dk=128, dv=128, pages=64, rows=16, width=3, forks=1),
        # 64 samples drawn from 16 prompts at once, 32 heads of 128 in 8 layers
        dict(name="fork 64", kind="fork", layers=8, H=32, dk=128, dv=128, pages=160, rows=128, width=4, forks=64),
        # a small pool with half its pages freed is packed
        dict(name="compact small", kind="compact", layers=2, H=8, dk=64, dv=64, pages=97, rows=48, width=2, live=45, movers=21),
        # a large pool is packed to hand memory back
        dict(name="compact large", kind="compact", layers=8, H=32, dk=128, dv=128, pages=160, rows=96, width=2, live=90,
             movers=40),
        # one chat's next token
        dict(name="decode one", kind="decode", B=1, pad=0, H=8, dk=128, dv=128, dtype="bf16", o="bf16", gate=False, pages=16),
        # a captured batch of 256 rows of which 6 are padding, 32 heads of 128
        dict(name="decode 256", kind="decode", B=256, pad=6, H=32, dk=128, dv=128, dtype="bf16", o="bf16", gate=False,
             pages=288),
        # one chat's draft of 8 tokens
        dict(name="verify one", kind="verify", B=1, H=8, K=8, dk=128, dv=128, depth=3, dtype="bf16", o="bf16", pages=16),
        # a batch of 64 chats with trees of up to 32 drafted tokens, verified and committed
        dict(name="step 64x32", kind="step", B=64, H=32, K=32, dk=128, dv=128, depth=6, dtype="bf16", o="bf16", pages=160),
        # deep ragged trees at full precision on half-size heads
        dict(name="step fp32 deep", kind="step", B=15, H=8, K=63, dk=64, dv=64, depth=12, dtype="f32", o="f32", pages=40),
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["heads", "heads", "fork", "compact", "decode", "verify", "step"])
    if kind == "heads":
        d = rng.choice([16, 32, 64, 96, 128, 192])
        hq = _log(rng, 1, 48)
        hk = rng.choice([hq, max(1, hq // 4), _log(rng, 1, 8)])
        n = _log(rng, 1, max(1, min(60000, (1 << 27) // ((hq + hk) * d))))
        rot = rng.choice([0, d if d % 16 == 0 else 0, 16])
        return dict(kind=kind, n=n, hq=hq, hk=hk, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), norm=rng.choice(["l2", "rms"]),
                    rot=rot, pairing=rng.choice(["halves", "pairs"]), fused=rng.random() < 0.5,
                    weights=rng.random() < 0.5, start=_log(rng, 1, 1000000))
    H = _log(rng, 1, 32)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 32), (32, 32), (16, 16)])
    page = 4 * H * dk * dv
    if kind == "fork":
        layers = rng.randint(1, 8)
        forks = _log(rng, 1, max(1, min(64, (500 << 20) // (page * layers))))
        rows = 2 * forks + rng.randint(1, 9)
        width = rng.randint(1, 4)
        return dict(kind=kind, layers=layers, H=H, dk=dk, dv=dv, pages=forks + 6 * width + rng.randint(1, 30) + 1, rows=rows,
                    width=width, forks=forks)
    if kind == "compact":
        layers = rng.randint(1, 8)
        live = _log(rng, 4, max(4, min(96, (900 << 20) // (page * layers))))
        movers = rng.randint(1, live // 2)
        return dict(kind=kind, layers=layers, H=H, dk=dk, dv=dv, pages=live + movers + rng.randint(0, 40),
                    rows=live + rng.randint(0, 9), width=rng.randint(1, 3), live=live, movers=movers)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    o = rng.choice(["bf16", "f32"])
    if kind == "decode":
        B = _log(rng, 1, max(1, min(512, (500 << 20) // page)))
        return dict(kind=kind, B=B, pad=rng.randint(0, B - 1) // 8, H=H, dk=dk, dv=dv, dtype=dtype, o=o, gate=rng.random() < 0.4,
                    pages=B + rng.randint(1, 20))
    K = _log(rng, 1, 64)
    B = _log(rng, 1, max(1, min(128, 2000 // H, 2000000 // (H * K * max(K, 32)))))
    return dict(kind=kind, B=B, H=H, K=K, dk=dk, dv=dv, depth=rng.randint(1, min(K, 12)), dtype=dtype, o=o,
                pages=2 * B + rng.randint(1, 9))


# ---- inputs ---------------------------------------------------------------------------------------


def _nodes(c, b):
    """How many nodes sequence b's tree has: the chain of `depth` nodes and, ragged, up to K."""
    return max(c["depth"], c["K"] - (b * 5) % (c["K"] // 4 + 1))


def _taken(c, b):
    """How many tokens of sequence b's drafts were accepted: 0 .. depth."""
    return (b + 1) % (c["depth"] + 1)


def _trees(c, g):
    """Parents [B][K]: nodes 0 .. depth-1 are a chain, each later one hangs below a random earlier one that
    is less than `depth` deep."""
    B, K, D = c["B"], c["K"], c["depth"]
    pick = torch.rand(B, K, generator=g)
    deep = torch.zeros(B, K, dtype=torch.int64)
    par = torch.full((B, K), -1, dtype=torch.int64)
    rows = torch.arange(B)
    for t in range(K):
        if t < D:
            p = torch.full((B,), t - 1)
        else:  # the r-th of the roots' level and the nodes that may have children
            may = torch.cat([torch.ones(B, 1), (deep[:, :t] < D).float()], 1)
            want = (pick[:, t] * may.sum(1)).floor() + 1
            p = (may.cumsum(1) >= want[:, None]).float().argmax(1) - 1
        par[:, t] = p
        deep[:, t] = torch.where(p >= 0, deep[rows, p.clamp(min=0)], torch.zeros(B, dtype=torch.int64)) + 1
    return par.to(torch.int32)


def _tokens(lead, H, dk, dv, dtype, g, dev):
    """q, unit keys, v, retentions and write strengths of the tokens [*lead][H]."""
    k = torch.randn(*lead, H, dk, generator=g, device=dev)
    k = k / k.norm(dim=-1, keepdim=True)
    return dict(q=torch.randn(*lead, H, dk, generator=g, device=dev).to(dtype), k=k.to(dtype),
                v=torch.randn(*lead, H, dv, generator=g, device=dev).to(dtype),
                alpha=torch.sigmoid(torch.randn(*lead, H, dk, generator=g, device=dev) + 3.0),
                beta=torch.sigmoid(torch.randn(*lead, H, generator=g, device=dev)))


def _ints(x, dev):
    return torch.as_tensor(x, dtype=torch.int32).to(dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = dict(c=c)
    if c["kind"] == "heads":
        n, hq, hk, d, dt = c["n"], c["hq"], c["hk"], c["d"], _DT[c["dtype"]]
        if c["fused"]:  # rows of a fused projection: queries, keys, and as many values
            row = torch.randn(n, hq + 2 * hk, d, generator=g, device=dev).to(dt)
            s["q"], s["k"] = row[:, :hq], row[:, hq:hq + hk]
        else:
            s["q"] = torch.randn(n, hq, d, generator=g, device=dev).to(dt)
            s["k"] = torch.randn(n, hk, d, generator=g, device=dev).to(dt)
        s["qo"], s["ko"] = torch.empty(n, hq, d, dtype=dt, device=dev), torch.empty(n, hk, d, dtype=dt, device=dev)
        s["qw"] = torch.rand(d, generator=g, device=dev) + 0.5 if c["weights"] else None
        s["kw"] = torch.rand(d, generator=g, device=dev) + 0.5 if c["weights"] else None
        s["pos"] = torch.arange(n, device=dev, dtype=torch.int32) + c["start"] if c["rot"] else None
        s["freq"] = (10000.0 ** (-torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) / max(1, c["rot"] // 2))).float() if c["rot"] else None
        s["eps"], s["scale"] = 1e-6, d ** -0.5
        return s
    if c["kind"] in ("fork", "compact"):
        L, P, R, W = c["layers"], c["pages"], c["rows"], c["width"]
        s["pool"] = torch.randn(L, P, c["H"], c["dk"], c["dv"], generator=g, device=dev)
        table, ref = torch.full((R, W), -1, dtype=torch.int64), torch.zeros(P, dtype=torch.int64)
        order = torch.randperm(P, generator=h)
        if c["kind"] == "fork":
            # a few prompts, each with its running state and the recorded states that its samples share
            prompts = min(max(1, c["forks"] // 4), (P - c["forks"]) // W, R - c["forks"])
            rows = torch.randperm(R, generator=h)
            table[rows[:prompts]] = order[:prompts * W].reshape(prompts, W)
            ref[order[:prompts * W]] = 1
            s["parents"] = _ints(rows[torch.randint(0, prompts, (c["forks"],), generator=h)], dev)
            s["children"] = _ints(rows[prompts:prompts + c["forks"]], dev)
            cap = c["forks"]
        else:
            live, m = c["live"], c["movers"]
            low, high = torch.randperm(live, generator=h)[m:], live + torch.randperm(P - live, generator=h)[:m]
            held = torch.cat([low, high])[torch.randperm(live, generator=h)]
            at = torch.randperm(R * W, generator=h)[:min(live, R * W)]
            table.view(-1)[at] = held[:len(at)]
            ref[held] = 1
            s["table_out"], s["ref_out"] = (torch.zeros(*x, dtype=torch.int32, device=dev) for x in ((R, W), (P,)))
            s["n_live"] = torch.zeros(1, dtype=torch.int32, device=dev)
            cap = P
        s["table"], s["ref"] = _ints(table, dev), _ints(ref, dev)
        s["moves"] = torch.zeros(cap, 2, dtype=torch.int32, device=dev)
        s["n_moves"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    B, H, dk, dv, P = c["B"], c["H"], c["dk"], c["dv"], c["pages"]
    s["pool"] = 0.1 * torch.randn(P, H, dk, dv, generator=g, device=dev)
    order = torch.randperm(P, generator=h)
    pages = order[:B].clone()
    if c["kind"] == "decode":
        pages[B - c["pad"]:] = -1
        s.update(_tokens((B,), H, dk, dv, _DT[c["dtype"]], g, dev))
        if c["gate"]:
            s["z"] = (-4.5 + 0.4 * torch.randn(B, H, dk, generator=g, device=dev)).to(_DT[c["dtype"]])
            s["A"] = 0.1 * torch.randn(H, generator=g, device=dev)
        s["o"] = torch.zeros(B, H, dv, dtype=_DT[c["o"]], device=dev)
    else:
        s.update(_tokens((B, c["K"]), H, dk, dv, _DT[c["dtype"]], g, dev))
        s["parents"] = _trees(c, h).to(dev)
        s["n_nodes"] = _ints([_nodes(c, b) for b in range(B)], dev)
        s["last"] = _ints([_taken(c, b) - 1 for b in range(B)], dev)
        s["pages_out"] = _ints(order[B:2 * B], dev) if c["kind"] == "step" else None
        s["o"] = torch.zeros(B, c["K"], H, dv, dtype=_DT[c["o"]], device=dev)
        s["u"] = torch.zeros(B, H, c["K"], dv, device=dev)
    s["pages"] = _ints(pages, dev)
    return s


# ---- one pass -------------------------------------------------------------------------------------


def run(state):
    return {"heads": _heads, "fork": _fork, "compact": _compact, "decode": _decode, "verify": _tree, "step": _tree}[state["c"]["kind"]](state)


def _head_norm(x, w, scale, s):
    """x [n][H][d] divided by its norm for each head, weighted, rotated by position."""
    c, x = s["c"], x.float()
    ss = (x * x).sum(-1, keepdim=True) if c["norm"] == "l2" else (x * x).mean(-1, keepdim=True)
    y = x / torch.sqrt(ss + s["eps"])
    if w is not None:
        y = y * w
    r = c["rot"]
    if r:
        angle = s["pos"].double()[:, None] * s["freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        if c["pairing"] == "halves":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        y = torch.cat([turned, y[..., r:]], -1)
    return y * scale


def _heads(s):
    c = s["c"]
    if own:
        import gated_delta_rule_07_amd as kda
        return list(kda.kda_qk_norm(s["q"], s["k"], norm=c["norm"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                                    q_scale=s["scale"], positions=s["pos"], inv_freq=s["freq"], pairing=c["pairing"],
                                    q_out=s["qo"], k_out=s["ko"]))
    return [_head_norm(s["q"], s["qw"], s["scale"], s).to(s["q"].dtype), _head_norm(s["k"], s["kw"], 1.0, s).to(s["k"].dtype)]


def _fork(s):
    """Children take over their parents' rows: slot 0, the running state, as a copy on a page of its own, the
    recorded states shared; then the children end and their pages are free again."""
    pool, table, ref = s["pool"], s["table"], s["ref"]
    if own:
        import gated_delta_rule_07_amd as kda
        moves, n = kda.kda_cache_fork(table, ref, s["parents"], s["children"], 1, moves=s["moves"], n_moves=s["n_moves"])
        kda.kda_cache_copy(pool, moves, n, n_layers=s["c"]["layers"])
        rows = table[s["children"]]
        kda.kda_cache_free(table, ref, s["children"])
        return [pool, rows, table, ref, moves, n]
    free = torch.sort((ref > 0).to(torch.int8), stable=True).indices  # free pages first, lowest first
    rows = table[s["parents"]]
    src, dst = rows[:, 0].clone(), free[:len(rows)].to(torch.int32)
    rows[:, 0] = dst
    table[s["children"]] = rows
    one = torch.ones(rows.numel(), dtype=torch.int32, device=ref.device)
    held = rows.flatten()
    ref.index_add_(0, held.clamp(min=0), one * (held >= 0))
    s["moves"].copy_(torch.stack([src, dst], 1))
    s["n_moves"].fill_(len(rows))
    pool[:, dst] = pool[:, src]
    rows = table[s["children"]]
    held = rows.flatten()
    ref.index_add_(0, held.clamp(min=0), -one * (held >= 0))
    table[s["children"]] = -1
    return [pool, rows, table, ref, s["moves"], s["n_moves"]]


def _compact(s):
    """Live pages move down into the free ones below them; the tables that name them follow."""
    pool, table, ref = s["pool"], s["table"], s["ref"]
    if own:
        import gated_delta_rule_07_amd as kda
        kda.kda_cache_compact(table, ref, table_out=s["table_out"], ref_out=s["ref_out"], moves=s["moves"],
                              n_moves=s["n_moves"], n_live=s["n_live"])
        kda.kda_cache_copy(pool, s["moves"], s["n_moves"], n_layers=s["c"]["layers"])
        return [pool, s["table_out"], s["ref_out"], s["moves"], s["n_moves"], s["n_live"]]
    held = ref > 0
    live = held.sum()
    at = torch.arange(len(ref), device=ref.device)
    src = torch.nonzero(held & (at >= live)).flatten()
    dst = torch.nonzero(~held & (at < live)).flatten()
    name = at.clone()
    name[src] = dst
    new = torch.where((table >= 0) & held[table.clamp(min=0)], name[table.clamp(min=0)], -1)
    s["table_out"].copy_(new)
    s["ref_out"].copy_(torch.where(held & (at < live), ref, 0))
    s["ref_out"][dst] = ref[src]
    s["moves"][:len(src)] = torch.stack([src, dst], 1).to(torch.int32)
    s["n_moves"].fill_(len(src))
    s["n_live"].copy_(live)
    pool[:, dst] = pool[:, src]
    return [pool, s["table_out"], s["ref_out"], s["moves"], s["n_moves"], s["n_live"]]


def _decode(s):
    """One step of the recurrence on each sequence's page; rows without a page are left as they were."""
    c, pool, pages, o = s["c"], s["pool"], s["pages"], s["o"]
    if own:
        import gated_delta_rule_07_amd as kda
        kda.kda_decode_step_paged(s["q"], s["k"], s["v"], None if c["gate"] else s["alpha"], s["beta"], pool, pages,
                                  z=s["z"] if c["gate"] else None, A=s["A"] if c["gate"] else None, o=o)
        return [o, pool]
    n = c["B"] - c["pad"]  # the padding of a batch stands at its end
    at = pages[:n]
    q, k, v, beta = s["q"][:n].float(), s["k"][:n].float(), s["v"][:n].float(), s["beta"][:n]
    alpha = torch.exp(-5.0 * torch.sigmoid(torch.exp(s["A"])[:, None] * s["z"][:n].float())) if c["gate"] else s["alpha"][:n]
    S = alpha[..., None] * pool[at]
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    pool[at] = S
    o[:n] = (S * q[..., None]).sum(-2).to(o.dtype)
    return [o, pool]


def _tree(s):
    """The recurrence along every path of a tree of drafted tokens; with pages_out, the state after the
    accepted path on another page."""
    c, pool = s["c"], s["pool"]
    step = c["kind"] == "step"
    if own:
        import gated_delta_rule_07_amd as kda
        o, u = kda.kda_tree_verify(s["q"], s["k"], s["v"], s["alpha"], s["beta"], pool, s["pages"], s["parents"], s["n_nodes"],
                                   o=s["o"], u=s["u"])
        if not step:
            return [o, u]
        kda.kda_tree_commit(s["k"], s["alpha"], u, s["parents"], s["last"], pool, s["pages"], s["pages_out"], s["n_nodes"])
        return [o, u, pool]
    B, K, H, dk, dv = c["B"], c["K"], c["H"], c["dk"], c["dv"]
    par, dev = s["parents"].long(), pool.device
    S0 = pool[s["pages"]]
    # above[b][t][r]: r is t or an ancestor of t
    above = torch.zeros(B, K, K, dtype=torch.bool, device=dev)
    here = torch.arange(K, device=dev).expand(B, K).contiguous()
    for _ in range(c["depth"]):
        above |= torch.arange(K, device=dev) == torch.where(here >= 0, here, -1)[..., None]
        here = torch.where(here >= 0, par.gather(1, here.clamp(min=0)), -1)
    head = lambda x: x.float().transpose(1, 2)  # noqa: E731  [B][K][H][d] -> [B][H][K][d]
    q, k, v, beta = head(s["q"]), head(s["k"]), head(s["v"]), s["beta"].transpose(1, 2)
    far = torch.matmul(above.double()[:, None], torch.log(head(s["alpha"]).double()))  # log decay from the root
    P = torch.exp(far).float()
    x, y = torch.matmul(P * k, S0), torch.matmul(P * q, S0)
    between = torch.where(above[:, None, :, :, None], (far[:, :, :, None] - far[:, :, None]), -math.inf).exp_().float()
    between = between * k[:, :, None]  # k_r, decayed from r to t
    cc = (between * k[:, :, :, None]).sum(-1).masked_fill(torch.eye(K, dtype=torch.bool, device=dev), 0.0)
    dd = (between * q[:, :, :, None]).sum(-1)
    u = beta[..., None] * (v - x)
    for _ in range(c["depth"] - 1):  # each turn makes one more level of the tree right
        u = beta[..., None] * (v - x - torch.matmul(cc, u))
    there = torch.arange(K, device=dev) < s["n_nodes"][:, None]
    s["u"].copy_(torch.where(there[:, None, :, None], u, s["u"]))
    s["o"].copy_(torch.where(there[:, :, None, None], (y + torch.matmul(dd, u)).transpose(1, 2).to(s["o"].dtype), s["o"]))
    if not step:
        return [s["o"], s["u"]]
    last = s["last"].long()
    rows = torch.arange(B, device=dev)
    path = (above[rows, last.clamp(min=0)] & (last >= 0)[:, None])[:, None, :, None]  # tokens that were accepted
    end = torch.where((last >= 0)[:, None, None], far[rows, :, last.clamp(min=0)], 0.0)[:, :, None]
    w = torch.where(path, end - far, -math.inf).exp().float() * k
    pool[s["pages_out"]] = torch.exp(end).float().transpose(-1, -2) * S0 + torch.matmul(w.transpose(-1, -2).contiguous(), u)
    return [s["o"], s["u"], pool]


# ---- what a pass cannot do without ----------------------------------------------------------------


def work(case):
    c = case
    if c["kind"] == "heads":
        vals = c["n"] * (c["hq"] + c["hk"]) * c["d"]
        more = 4 * c["n"] + 2 * c["rot"] if c["rot"] else 0
        return dict(bytes=2 * vals * (2 if c["dtype"] == "bf16" else 4) + more + (8 * c["d"] if c["weights"] else 0),
                    flops=vals * (4 + (3 if c["rot"] else 0)))
    page = 4 * c["H"] * c["dk"] * c["dv"]
    if c["kind"] == "fork":
        return dict(bytes=2 * page * c["layers"] * c["forks"] + 4 * (c["pages"] + 6 * c["forks"] * c["width"]), flops=0)
    if c["kind"] == "compact":
        return dict(bytes=2 * page * c["layers"] * c["movers"] + 8 * (c["pages"] + c["rows"] * c["width"]), flops=0)
    e, eo = (2 if c["dtype"] == "bf16" else 4), (2 if c["o"] == "bf16" else 4)
    H, dk, dv = c["H"], c["dk"], c["dv"]
    if c["kind"] == "decode":
        n = c["B"] - c["pad"]
        row = H * (e * (2 * dk + dv) + (e if c["gate"] else 4) * dk + 4 + eo * dv)
        return dict(bytes=n * (2 * page + row), flops=n * H * 7 * dk * dv)
    nodes = sum(_nodes(c, b) for b in range(c["B"]))
    row = H * (e * (2 * dk + dv) + 4 * dk + 4 + eo * dv + 4 * dv)
    got = dict(bytes=c["B"] * page + nodes * row, flops=nodes * H * 4 * dk * dv)
    if c["kind"] == "step":
        taken = sum(_taken(c, b) for b in range(c["B"]))
        got["bytes"] += 2 * c["B"] * page + taken * H * ((e + 4) * dk + 4 * dv)
        got["flops"] += (c["B"] + 2 * taken) * H * dk * dv
    return got


# ---- the definitions, in 64 bits ------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, torch.device("cuda")
    if c["kind"] == "heads":
        out = []
        for x, w, scale in ((s["q"], s["qw"], s["scale"]), (s["k"], s["kw"], 1.0)):
            x = x.double()
            size = x.pow(2).sum(-1)
            if c["norm"] == "rms":
                size = size / c["d"]
            x *= (scale * (size + s["eps"]).rsqrt())[..., None]
            if w is not None:
                x *= w.double()
            r = c["rot"]
            if r:  # each pair as a complex number, turned
                i = torch.arange(r // 2, device=dev)
                a, b = (i, i + r // 2) if c["pairing"] == "halves" else (2 * i, 2 * i + 1)
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), s["pos"].double()[:, None] * s["freq"].double()[None])
                pair = torch.complex(x[..., a], x[..., b]) * turn[:, None]
                x[..., a], x[..., b] = pair.real, pair.imag
            out.append(x)
        return out
    if c["kind"] in ("fork", "compact"):
        pool, table, ref = s["pool"].double(), s["table"].tolist(), s["ref"].tolist()
        moves, rows = [], []
        if c["kind"] == "fork":
            for p, _ in zip(s["parents"].tolist(), s["children"].tolist()):
                page = ref.index(0)
                ref[page] = 1
                moves.append((table[p][0], page))
                rows.append([page] + table[p][1:])
            for a, b in moves:
                pool[:, b] = pool[:, a]
            return [pool, _ints(rows, dev), s["table"], s["ref"], _ints(moves, dev), _ints([len(moves)], dev)]
        live = sum(r > 0 for r in ref)
        holes = [p for p in range(live) if ref[p] == 0]
        for p in range(live, c["pages"]):
            if ref[p] > 0:
                moves.append((p, holes[len(moves)]))
        name = {p: p for p in range(live)} | dict(moves)
        for a, b in moves:
            pool[:, b] = pool[:, a]
            ref[b], ref[a] = ref[a], 0
        listed_moves = moves + [(0, 0)] * (c["pages"] - len(moves))
        return [pool, _ints([[name.get(p, -1) for p in r] for r in table], dev), _ints(ref, dev), _ints(listed_moves, dev),
                _ints([len(moves)], dev), _ints([live], dev)]
    x = {n: s[n].double() for n in ("q", "k", "v", "alpha", "beta", "pool")}
    pages = s["pages"].long()
    if c["kind"] == "decode":
        if c["gate"]:
            x["alpha"] = torch.exp(-5 / (1 + torch.exp(-torch.exp(s["A"].double())[None, :, None] * s["z"].double())))
        o = s["o"].double()
        for b in range(c["B"] - c["pad"]):
            S = x["pool"][pages[b]] * x["alpha"][b, :, :, None]
            S += x["beta"][b, :, None, None] * x["k"][b, :, :, None] * (x["v"][b] - (x["k"][b, :, None] @ S)[:, 0])[:, None]
            x["pool"][pages[b]] = S
            o[b] = (x["q"][b, :, None] @ S)[:, 0]
        return [o, x["pool"]]
    o, u = s["o"].double(), s["u"].double()
    for b in range(c["B"]):  # every node's own state, one token after another
        par, first = s["parents"][b].tolist(), x["pool"][pages[b]].clone()
        states = []
        for t in range(_nodes(c, b)):
            S = (states[par[t]] if par[t] >= 0 else first) * x["alpha"][b, t, :, :, None]
            write = x["beta"][b, t, :, None] * (x["v"][b, t] - (x["k"][b, t, :, None] @ S)[:, 0])
            S = S + x["k"][b, t, :, :, None] * write[:, None]
            u[b, :, t], o[b, t] = write, (x["q"][b, t, :, None] @ S)[:, 0]
            states.append(S)
        if c["kind"] == "step":
            last = _taken(c, b) - 1
            x["pool"][int(s["pages_out"][b])] = states[last] if last >= 0 else first
    return [o, u] + ([x["pool"]] if c["kind"] == "step" else [])
