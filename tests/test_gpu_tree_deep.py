"""Deep trees against the recurrence in 64 bits, with bounds that stay small at every depth (tree_bounds): o, u and the
committed states of chains of 64 and of trees as deep."""
import numpy as np
import pytest
import torch

import kda_inputs as ki
import serving_model as sm
import tree_bounds as tb
from test_tree_bounds import TREES

pytestmark = pytest.mark.gpu


def _host(x):
    return x.detach().double().cpu().numpy()


@pytest.mark.parametrize("o_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype,dk,dv", [(torch.bfloat16, 128, 128), (torch.float32, 128, 128), (torch.float32, 64, 16),
                                         (torch.bfloat16, 16, 32), (torch.float32, 32, 64), (torch.bfloat16, 64, 128)])
def test_deep_trees(gpu, dtype, dk, dv, o_dtype):
    import gated_delta_rule_07_amd as kda
    trees = list(TREES.values())
    lasts = [[63, 62, 63, 63], [31, 47, 40, 33], [48, 63, 15, 50]]
    B, K, H = len(trees), 64, 2
    d = ki.make_prefill(B, K, H, dk, dv, dtype, 3.0, 0.1, seed=21, device=gpu)
    d.pop("S0")
    pool = ki.make_state(2 * B, H, dk, dv, 0.1, 22, gpu)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    par = ints(trees)
    ins, outs = list(range(B)), list(range(B, 2 * B))
    o, u = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, ints(ins), par, o_dtype=o_dtype)
    got = []
    for last in lasts:
        kda.kda_tree_commit(d["k"], d["alpha"], u, par, ints(last), pool, ints(ins), ints(outs))
        got.append(_host(pool)[B:])
    x, ho, hu, hp = {n: _host(t) for n, t in d.items()}, _host(o), _host(u), _host(pool)
    hs = sm.HALF_STEP["bf16" if o_dtype == torch.bfloat16 else "f32"]
    for b in range(B):
        for h in range(H):
            row = [x[n][b, :, h] for n in ("q", "k", "v", "alpha", "beta")]
            r = sm.tree_run(hp[b, h], *row, trees[b])
            eo, eu, es = tb.bounds(hp[b, h], *row, trees[b], r["u"])
            sm.within(ho[b, :, h], r["o"], eo, hs, f"o of ({b}, {h})")
            sm.within(hu[b, h], r["u"], eu, sm.U, f"u of ({b}, {h})")
            for last, state in zip(lasts, got):
                sm.within(state[b, h], r["states"][last[b]], es(last[b]), sm.U, f"state of ({b}, {h}) after node {last[b]}")
