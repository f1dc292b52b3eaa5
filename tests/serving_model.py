"""Plain models of the serving operators, for the tests: 64-bit arithmetic on the host, one step after another,
sharing nothing with the library.  The numeric ones also give a bound on what fp32 arithmetic may differ by."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the output's type, relative


# ---- norms of queries and keys --------------------------------------------------------------------


def head_norm(x, norm, eps, weight=None, scale=1.0, positions=None, inv_freq=None, pairing="halves"):
    """(y, slack) for x [n][H][d] in float64: the formula, and what fp32 may be off before the last rounding.

    A value is a product of x with a norm, a weight and a scale.  The norm's sum of d squares takes at most
    13 additions in a row (8 in a lane, 5 across 32 lanes) and one product, half of which the root halves; the
    division by d, adding eps, the root, the quotient, and the two products with weight and scale add a step
    each: under 16 u of the value.  A rotation adds two products, a sum, and the errors of the
    cosine and sine: 4 u each for the function and the angle's rounding to fp32 after its reduction to a
    fraction of a turn (an angle within pi: at most 2 pi u = 7 u), and an fp64 angle of up to 2^31 turns
    times 2^-52 (another 2^-21 = 8 u): under 32 u of |a| + |b|.  Together below 64 u."""
    x = x.astype(np.float64)
    with np.errstate(all="ignore"):
        ss = (x * x).sum(-1, keepdims=True)
        if norm == "rms":
            ss = ss / x.shape[-1]
        y = x / np.sqrt(ss + eps)
        if weight is not None:
            y = y * weight.astype(np.float64)
        size = np.abs(y)
        if inv_freq is not None and len(inv_freq):
            r = 2 * len(inv_freq)
            f = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
            c, s = np.cos(f)[:, None], np.sin(f)[:, None]
            i = np.arange(r // 2)
            a, b = (i, i + r // 2) if pairing == "halves" else (2 * i, 2 * i + 1)
            ya, yb = y[..., a].copy(), y[..., b].copy()
            y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
            both = np.abs(ya) + np.abs(yb)
            size[..., a], size[..., b] = both, both
    return y * scale, 64 * U * size * abs(scale)


# ---- the cache of state pages ---------------------------------------------------------------------


def _holds(page, n_pages):
    return 0 <= page < n_pages


def fork(table, ref, parents, children, n_private):
    """Applies kda_cache_fork's rules to lists; returns (table, ref, moves)."""
    table, ref, P, R = [list(r) for r in table], list(ref), len(ref), len(table)
    before = [list(r) for r in table]
    empty = [not any(_holds(p, P) for p in r) for r in before]
    free = [p for p in range(P) if ref[p] <= 0]
    moves, named, short = [], set(), False
    for par, ch in zip(parents, children):
        if not (0 <= ch < R and -1 <= par < R) or ch in named:
            continue
        named.add(ch)
        if not empty[ch]:
            continue
        row = [-1] * len(before[0]) if par < 0 else before[par]
        take = [w for w in range(n_private) if par < 0 or _holds(row[w], P)]
        if short or len(take) > len(free):
            short = True
            continue
        new = []
        for w, page in enumerate(row):
            if w in take:
                to = free.pop(0)
                moves.append((page if par >= 0 else -1, to))
                ref[to] = 1
                new.append(to)
            elif w >= n_private and _holds(page, P):
                ref[page] += 1
                new.append(page)
            else:
                new.append(-1)
        table[ch] = new
    return table, ref, moves


def free(table, ref, rows):
    table, ref = [list(r) for r in table], list(ref)
    for r in rows:
        if 0 <= r < len(table):
            for w, page in enumerate(table[r]):
                if _holds(page, len(ref)) and ref[page] > 0:
                    ref[page] -= 1
                table[r][w] = -1
    return table, ref


def compact(table, ref):
    """(table, ref, moves, n_live) after packing."""
    live = [p for p in range(len(ref)) if ref[p] > 0]
    holes = [p for p in range(len(live)) if ref[p] <= 0]
    movers = [p for p in live if p >= len(live)]
    name = {p: p for p in live}
    name.update(zip(movers, holes))
    out = [0] * len(ref)
    for p in live:
        out[name[p]] = ref[p]
    return [[name.get(p, -1) for p in r] for r in table], out, list(zip(movers, holes)), len(live)


def copy(src, dst, moves, same):
    """dst [layers][pages][...] after the moves that do not race."""
    out = dst.copy()
    n_src, n_dst = src.shape[1], dst.shape[1]
    good = [(a, b) for a, b in moves if _holds(b, n_dst) and (a == -1 or _holds(a, n_src)) and not (same and a == b)]
    targets = [b for _, b in good]
    for a, b in good:
        if targets.count(b) > 1 or (same and a >= 0 and a in targets):
            continue
        out[:, b] = 0 if a < 0 else src[:, a]
    return out


def runs(pages_in, pages_out, n_pages):
    """Which sequences of a call on pages run: valid pages, none of which another valid sequence writes."""
    ok = [_holds(i, n_pages) and _holds(o, n_pages) for i, o in zip(pages_in, pages_out)]
    return [ok[b] and not any(j != b and ok[j] and pages_out[j] in (pages_in[b], pages_out[b]) for j in range(len(ok)))
            for b in range(len(ok))]


# ---- trees ----------------------------------------------------------------------------------------


def tree_run(S, q, k, v, alpha, beta, parents):
    """One (sequence, head): every node's own state, in float64.

    S [dk][dv]; q, k, alpha [K][dk]; v [K][dv]; beta [K]; parents [K].  Returns dict of o, u [K][dv], states
    [K][dk][dv], and a bound on fp32's error of each.  The bound: the same recurrence on absolute values
    dominates every intermediate; each node's products sum at most d_k + 2 depth terms of at most 4 factors
    and each level passes on the errors of the ones above it, so (depth + 1) (d_k + 2 depth + 16) roundings of u
    times the dominating value."""
    K, dk = k.shape
    f = lambda a: np.asarray(a, dtype=np.float64)  # noqa: E731
    S, q, k, v, alpha, beta = map(f, (S, q, k, v, alpha, beta))
    states, big, o, u, eo, eu, es, depth = [], [], [], [], [], [], [], []
    for t in range(K):
        p = parents[t]
        dep = depth[p] + 1 if p >= 0 else 1
        Sb = alpha[t][:, None] * (states[p] if p >= 0 else S)
        Bb = alpha[t][:, None] * (big[p] if p >= 0 else np.abs(S))
        ut = beta[t] * (v[t] - Sb.T @ k[t])
        bu = np.abs(beta[t]) * (np.abs(v[t]) + Bb.T @ np.abs(k[t]))
        St, Bt = Sb + np.outer(k[t], ut), Bb + np.outer(np.abs(k[t]), bu)
        n = (dep + 1) * (dk + 2 * dep + 16) * U
        states.append(St)
        big.append(Bt)
        o.append(St.T @ q[t])
        u.append(ut)
        eo.append(n * (Bt.T @ np.abs(q[t])))
        eu.append(n * bu)
        es.append(n * Bt)
        depth.append(dep)
    return dict(o=np.stack(o), u=np.stack(u), states=np.stack(states), eo=np.stack(eo), eu=np.stack(eu), es=np.stack(es),
                depth=depth)


def fix_parents(parents):
    """Parents as the library reads them: a value outside [-1, t) is -1."""
    return [p if -1 <= p < t else -1 for t, p in enumerate(parents)]


def random_tree(rng, K, depth):
    """Parents of K nodes, at most `depth` deep."""
    par, deep = [], []
    for t in range(K):
        may = [-1] + [s for s in range(t) if deep[s] < depth]
        p = int(rng.choice(may))
        par.append(p)
        deep.append(deep[p] + 1 if p >= 0 else 1)
    return par


def within(got, ref, slack, half_step, what=""):
    """got (any float array) is the rounding of a value within slack of ref; NaN never passes."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    tol = slack + half_step * (np.abs(ref) + slack) + 1e-37
    off = np.abs(got - ref)
    bad = ~(off <= tol)
    worst = float(np.nanmax(off / tol)) if off.size else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values off, worst {worst:.3g} of the bound"
    return worst
