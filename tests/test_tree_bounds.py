"""CPU checks of tree_bounds: small enough at every depth that a wrong value fails, and wide enough for fp32 arithmetic
of another order than the kernel's."""
import numpy as np
import pytest
import torch

import kda_inputs as ki
import serving_model as sm
import tree_bounds as tb

TREES = {"chain": list(range(-1, 63)), "two chains": [max(-1, t - 2) for t in range(64)],
         "binary": [(t - 1) // 2 if t else -1 for t in range(64)], "random": sm.random_tree(np.random.default_rng(3), 64, 64)}
SHAPES = [(torch.bfloat16, 128, 128), (torch.float32, 128, 64), (torch.float32, 64, 16), (torch.bfloat16, 16, 32)]


def _inputs(dtype, dk, dv, seed=7):
    d = ki.make_prefill(1, 64, 1, dk, dv, dtype, 3.0, 0.1, seed=seed)
    x = {n: t.double().numpy()[0, :, 0] for n, t in d.items() if n != "S0"}
    return d["S0"].double().numpy()[0, 0], x


def _rms(a):
    return np.sqrt(np.mean(a * a, -1, keepdims=True))


@pytest.mark.parametrize("tree", TREES)
@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
def test_bounds_stay_small_at_every_depth(tree, dtype, dk, dv):
    """Below a fiftieth of each row's rms, so zeros, a sign, or a term left out cannot pass."""
    S, x = _inputs(dtype, dk, dv)
    par = TREES[tree]
    r = sm.tree_run(S, *(x[n] for n in ("q", "k", "v", "alpha", "beta")), par)
    eo, eu, es = tb.bounds(S, *(x[n] for n in ("q", "k", "v", "alpha", "beta")), par, r["u"])
    assert (eo <= 0.02 * _rms(r["o"])).all() and (eu <= 0.02 * _rms(r["u"])).all()
    for last in (15, 31, 47, 63):
        assert (es(last) <= 0.02 * _rms(r["states"][last].ravel())).all()


@pytest.mark.parametrize("tree", TREES)
@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
def test_fp32_recurrence_lies_within_the_bounds(tree, dtype, dk, dv):
    """The recurrence in fp32, node after node, against the one in 64 bits; and mistakes in the last half of the tree
    (planted here, in the copy that is compared) lie outside."""
    S, x = _inputs(dtype, dk, dv)
    par = TREES[tree]
    q, k, v, al, be = (x[n] for n in ("q", "k", "v", "alpha", "beta"))
    r = sm.tree_run(S, q, k, v, al, be, par)
    eo, eu, es = tb.bounds(S, q, k, v, al, be, par, r["u"])
    f = np.float32
    states, o, u = [], [], []
    for t in range(64):
        Sb = f(al[t])[:, None] * (states[par[t]] if par[t] >= 0 else f(S))
        ut = f(be[t]) * (f(v[t]) - Sb.T @ f(k[t]))
        states.append(Sb + np.outer(f(k[t]), ut))
        o.append(states[t].T @ f(q[t]))
        u.append(ut)
    o, u = np.stack(o), np.stack(u)
    sm.within(o, r["o"], eo, sm.U, "o")
    sm.within(u, r["u"], eu, sm.U, "u")
    for last in (31, 63):
        sm.within(states[last], r["states"][last], es(last), sm.U, "state")
    for t in (33, 63):
        for wrong in (np.zeros_like(o[t]), -o[t], o[t] * 1.05):
            with pytest.raises(AssertionError):
                sm.within(wrong, r["o"][t], eo[t], sm.HALF_STEP["bf16"])


@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
def test_equations_of_the_nodes_are_the_recurrence(dtype, dk, dv):
    """The equations that the bounds start from give tree_run's outputs (in 64 bits)."""
    S, x = _inputs(dtype, dk, dv, seed=9)
    q, k, v, al, be = (x[n] for n in ("q", "k", "v", "alpha", "beta"))
    par = TREES["random"]
    r = sm.tree_run(S, q, k, v, al, be, par)
    for t in range(64):
        P, g, path = al[t].copy(), al[t].copy(), par[t]
        xt, ot = np.zeros(dv), (k[t] @ q[t]) * r["u"][t]
        while path >= 0:
            xt, ot = xt + (k[path] * g) @ k[t] * r["u"][path], ot + (k[path] * g) @ q[t] * r["u"][path]
            g, P, path = g * al[path], P * al[path], par[path]
        assert np.allclose(be[t] * (v[t] - S.T @ (P * k[t]) - xt), r["u"][t], rtol=0, atol=1e-12)
        assert np.allclose(S.T @ (P * q[t]) + ot, r["o"][t], rtol=0, atol=1e-11)
