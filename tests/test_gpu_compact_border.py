"""kda_cache_compact on both sides of the table size from which its entries are renamed by a launch of their own."""
import random

import pytest
import torch

import serving_model as sm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,W", [(1023, 1), (1025, 1), (2047, 1), (1024, 2), (1, 2048), (2049, 1), (683, 3), (1024, 8), (8193, 1)])
def test_tables_around_the_border(gpu, R, W, in_place):
    import gated_delta_rule_07_amd as kda
    rng = random.Random(R + W)
    P = 1500
    ref = [rng.randint(1, 3) if rng.random() < 0.4 else -rng.randint(0, 1) for _ in range(P)]
    table = [[rng.randint(-2, P) for _ in range(W)] for _ in range(R)]
    t, f = (torch.tensor(x, dtype=torch.int32, device=gpu) for x in (table, ref))
    to, fo, moves, n, live = kda.kda_cache_compact(t, f, table_out=t if in_place else None, ref_out=f if in_place else None)
    wt, wf, wm, wl = sm.compact(table, ref)
    assert int(live) == wl and [tuple(m) for m in moves[:int(n)].tolist()] == wm
    assert to.tolist() == wt and fo.tolist() == wf
