"""Trees one path of which grows past fp32's range from finite inputs: nodes that do not follow it keep their bounds.

Keys are taken as they are given, so a path that repeats a long key multiplies its write vectors by up to
beta |k|^2 - 1 a node and leaves fp32 after some nodes; the nodes beside it, and those above the overflow, are ordinary
numbers, and their outputs are those of the recurrence along their own paths."""
import numpy as np
import pytest
import torch

import kda_inputs as ki
import serving_model as sm

pytestmark = pytest.mark.gpu


def _host(x):
    return x.detach().double().cpu().numpy()


def _chain_beside(K, chain, first, rng):
    """Parents: a chain of `chain` nodes whose t-th node is node first + 2 t while room lasts (roots and their children
    between them), the other nodes independent roots or children of such roots."""
    at = [first + 2 * t for t in range(chain) if first + 2 * t < K]
    rest = [t for t in range(K) if t not in at]
    for t in rest:  # (what does not fit between goes where there is room)
        if len(at) == chain:
            break
        if t > first:
            at.append(t)
    at = sorted(at[:chain])
    par, roots = [-1] * K, []
    for t in range(K):
        if t in at:
            i = at.index(t)
            par[t] = at[i - 1] if i else -1
        else:
            par[t] = int(rng.choice(roots)) if roots and rng.random() < 0.4 else -1
            roots.append(t)
    return par, at


TREES = [  # K, nodes of the chain, its first node, norm of its one key (0: another key each node), beta, alpha
    (64, 48, 0, 8.0, 0.9, 0.97),
    (64, 30, 3, 8.0, 0.9, 0.97),
    (30, 14, 0, 1100.0 ** 0.5, 0.95, 0.999),
    (16, 12, 0, 100.0, 0.9, 0.97),
    (16, 6, 1, 1e4, 0.999, 0.999),
    (33, 6, 20, 1e8, 0.999, 0.999),
    (64, 40, 0, -20.0, 0.9, 0.97),  # (a key of norm 20 of its own for each node)
]


@pytest.mark.parametrize("K,chain,first,size,beta,alpha", TREES)
@pytest.mark.parametrize("dtype,dk,dv", [(torch.float32, 64, 64), (torch.bfloat16, 128, 128), (torch.float32, 128, 16)])
def test_a_path_that_overflows_stays_by_itself(gpu, K, chain, first, size, beta, alpha, dtype, dk, dv):
    import gated_delta_rule_07_amd as kda
    rng = np.random.default_rng(K + chain)
    d = ki.make_prefill(2, K, 1, dk, dv, dtype, 3.0, 0.1, seed=K, device=gpu)
    pool = ki.make_state(2, 1, dk, dv, 0.1, 9, gpu)
    par, at = _chain_beside(K, chain, first, rng)
    parents = [par, sm.random_tree(rng, K, 5)]
    k = d["k"].float()
    if size > 0:
        k[0, at] = size * k[0, at[0]].clone()
    else:
        k[0, at] *= -size
    d["k"] = k.to(dtype)
    d["beta"][0, at], d["alpha"][0, at] = beta, alpha
    assert all(bool(torch.isfinite(t.float()).all()) for t in d.values())
    o, u = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, None,
                               torch.tensor(parents, dtype=torch.int32, device=gpu))
    x, ho, hu, hp = {n: _host(t) for n, t in d.items()}, _host(o), _host(u), _host(pool)
    for b in range(2):
        with np.errstate(all="ignore"):
            r = sm.tree_run(hp[b, 0], *(x[n][b, :, 0] for n in ("q", "k", "v", "alpha", "beta")), parents[b])
        # the same recurrence on absolute values bounds every intermediate; a node whose bound lies well inside
        # fp32's range has to be right
        roundings = np.array([(dep + 1) * (dk + 2 * dep + 16) * sm.U for dep in r["depth"]])[:, None]
        inside = ((r["eo"] / roundings < 1e36) & (r["eu"] / roundings < 1e36)).all(1)
        beside = [t for t in range(K) if b == 1 or t not in at]
        assert inside[beside].all()
        if b == 0:
            assert 0 < inside[at].sum() < len(at), "the chain has to leave fp32's range on its way"
        sm.within(ho[b, inside, 0], r["o"][inside], r["eo"][inside], sm.U, "o")
        sm.within(hu[b, 0][inside], r["u"][inside], r["eu"][inside], sm.U, "u")
