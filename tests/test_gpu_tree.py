"""kda_tree_verify and kda_tree_commit against the recurrence run along every path in 64 bits.

The bounds are those of fp32 arithmetic (see serving_model.tree_run) and half a step of o's type."""
import random

import numpy as np
import pytest
import torch

import kda_inputs as ki
import serving_model as sm

pytestmark = pytest.mark.gpu


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _host(x):
    return x.detach().double().cpu().numpy()


def _drafts(gpu, B, K, H, dk, dv, dtype, P, seed):
    d = ki.make_prefill(B, K, H, dk, dv, dtype, 3.0, 0.1, seed=seed, device=gpu)
    d.pop("S0")
    return d, ki.make_state(P, H, dk, dv, 0.1, seed + 1, gpu)


def _check(gpu, d, pool, pages, parents, nodes=None, o_dtype=torch.float32, last=None, outs=None):
    """verify (and commit, with `last`) and every value of the outputs and the pool."""
    kda = _kda()
    B, K, H, dk = d["q"].shape
    dv = d["v"].shape[-1]
    o = torch.full((B, K, H, dv), 9.0, device=gpu, dtype=o_dtype)
    u = torch.full((B, H, K, dv), 9.0, device=gpu)
    before = pool.clone()
    tp, tn = _i(parents, gpu), None if nodes is None else _i(nodes, gpu)
    tpages = None if pages is None else _i(pages, gpu)
    kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, tpages, tp, tn, o=o, u=u)
    torch.cuda.synchronize()
    assert torch.equal(pool, before), "verify wrote the pool"
    ins = list(range(B)) if pages is None else pages
    x = {n: _host(t) for n, t in d.items()}
    ho, hu, hp = _host(o), _host(u), _host(pool)
    hs = sm.HALF_STEP["bf16" if o_dtype == torch.bfloat16 else "f32"]
    ref = {}
    for b in range(B):
        n = K if nodes is None else min(max(nodes[b], 0), K)
        if not 0 <= ins[b] < pool.shape[0]:
            n = 0
        assert (ho[b, n:] == 9.0).all() and (hu[b, :, n:] == 9.0).all(), f"sequence {b}: rows behind its tree were written"
        for h in range(H):
            if n == 0:
                continue
            r = ref[b, h] = sm.tree_run(hp[ins[b], h], x["q"][b, :n, h], x["k"][b, :n, h], x["v"][b, :n, h], x["alpha"][b, :n, h],
                                        x["beta"][b, :n, h], sm.fix_parents(parents[b])[:n])
            sm.within(ho[b, :n, h], r["o"], r["eo"], hs, f"o of ({b}, {h})")
            sm.within(hu[b, h, :n], r["u"], r["eu"], sm.U, f"u of ({b}, {h})")
    if last is None:
        return o, u
    kda.kda_tree_commit(d["k"], d["alpha"], u, tp, _i(last, gpu), pool, tpages, None if outs is None else _i(outs, gpu), tn)
    torch.cuda.synchronize()
    got, touched = _host(pool), set()
    to = ins if outs is None else outs
    for b, go in enumerate(sm.runs(ins, to, pool.shape[0])):
        if not go:
            continue
        n = K if nodes is None else min(max(nodes[b], 0), K)
        touched.add(to[b])
        for h in range(H):
            if not 0 <= last[b] < n:
                assert np.array_equal(got[to[b], h], hp[ins[b], h]), f"sequence {b}: nothing accepted"
            else:
                r = ref[b, h]
                sm.within(got[to[b], h], r["states"][last[b]], r["es"][last[b]], sm.U, f"state of ({b}, {h})")
    for page in range(pool.shape[0]):
        if page not in touched:
            assert np.array_equal(got[page], hp[page]), f"page {page} was written"
    return o, u


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_head_sizes(gpu, dtype, dk, dv):
    rng = np.random.default_rng(dk + dv)
    B, H, K = 2, 2, 21
    d, pool = _drafts(gpu, B, K, H, dk, dv, dtype, 5, dk + dv)
    parents = [sm.random_tree(rng, K, 6) for _ in range(B)]
    _check(gpu, d, pool, [4, 1], parents, last=[20, 13], outs=[0, 1])


@pytest.mark.parametrize("K", [1, 2, 3, 15, 16, 17, 31, 32, 33, 47, 48, 49, 57, 63, 64])
def test_sizes_of_trees(gpu, K):
    rng = np.random.default_rng(K)
    d, pool = _drafts(gpu, 2, K, 1, 128, 128, torch.bfloat16, 3, K)
    parents = [sm.random_tree(rng, K, 8), sm.random_tree(rng, K, 64)]
    _check(gpu, d, pool, [2, 0], parents, last=[K - 1, K // 2])


@pytest.mark.parametrize("dtype,dk,dv", [(torch.bfloat16, 128, 128), (torch.float32, 128, 128), (torch.float32, 64, 16)])
def test_shapes_of_trees(gpu, dtype, dk, dv):
    """A chain of 64, a star, two chains, a full binary tree, and parents that are not allowed (read as the root)."""
    K = 64
    chain, star = list(range(-1, K - 1)), [-1] * K
    two = [max(-1, t - 2) for t in range(K)]
    binary = [(t - 1) // 2 if t else -1 for t in range(K)]
    wrong = [t if t % 3 == 0 else (-5 if t % 3 == 1 else (t - 1 if t % 2 else 2 ** 31 - 1)) for t in range(K)]
    trees = [chain, star, two, binary, wrong]
    d, pool = _drafts(gpu, 5, K, 1, dk, dv, dtype, 6, 77)
    _check(gpu, d, pool, [5, 4, 3, 2, 1], trees, last=[63, 5, 62, 40, 11])


def test_ragged_trees_and_padding(gpu):
    """Trees of 0 to more than K nodes (clamped), sequences without a page, last nodes out of range, copies of a
    state onto another page where nothing was accepted."""
    rng = np.random.default_rng(4)
    B, K, H = 9, 20, 2
    d, pool = _drafts(gpu, B, K, H, 64, 64, torch.bfloat16, 20, 8)
    parents = [sm.random_tree(rng, K, 5) for _ in range(B)]
    nodes = [0, 1, 5, 20, 33, -2, 16, 17, 20]
    pages = [0, 1, -1, 3, 4, 5, 20, 7, 8]
    last = [0, 0, 2, 20, 19, 3, 1, -1, -1]
    _check(gpu, d, pool.clone(), pages, parents, nodes, torch.bfloat16, last=last)
    _check(gpu, d, pool.clone(), pages, parents, nodes, torch.float32, last=last, outs=[10, 11, 12, 13, 14, 15, 16, 17, 18])


def test_pages_left_out(gpu):
    """No page list: page b; commits that would race are passed over."""
    rng = np.random.default_rng(5)
    B, K = 6, 7
    d, pool = _drafts(gpu, B, K, 2, 32, 32, torch.float32, 9, 3)
    parents = [sm.random_tree(rng, K, 4) for _ in range(B)]
    _check(gpu, d, pool.clone(), None, parents, last=[6, 5, 4, 3, 2, 1])
    _check(gpu, d, pool.clone(), [0, 0, 1, 2, 3, 3], parents, last=[6, 5, 4, 3, 2, 1], outs=[6, 7, 1, 8, 8, 4])
    _check(gpu, d, pool.clone(), [0, 0, 1, 2, 2, 3], parents, last=[6, 5, 4, 3, 2, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steep_decay(gpu, dtype):
    """Decays that wipe a channel (0), or pass fp32's range over the path: products along the path, no quotients."""
    rng = np.random.default_rng(6)
    B, K, H = 2, 40, 2
    d, pool = _drafts(gpu, B, K, H, 128, 32, dtype, 4, 13)
    a = d["alpha"].clone()
    a[:, 2, :, 0::7] = 0.0
    a[:, 5, :, 1::5] = 1e-30
    a[:, :, :, 3::4] = 2.0 ** -20
    a[1, :, 1, :] = 2.0 ** -20
    d["alpha"] = a.contiguous()
    _check(gpu, d, pool, [3, 1], [sm.random_tree(rng, K, 40), list(range(-1, K - 1))], last=[39, 39])


def test_a_chain_equals_the_chain_calls(gpu):
    """A tree that is a chain of 16, on a dense state, agrees with kda_decode_verify and kda_decode_commit."""
    kda = _kda()
    B, K, H = 3, 16, 4
    d, S = _drafts(gpu, B, K, H, 128, 128, torch.bfloat16, B, 5)
    S2 = S.clone()
    o, u = kda.kda_decode_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], S)
    kda.kda_decode_commit(d["k"], d["alpha"], u, _i([16, 7, 0], gpu), S)
    par = _i([list(range(-1, K - 1))] * B, gpu)
    o2, u2 = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], S2, None, par)
    kda.kda_tree_commit(d["k"], d["alpha"], u2, par, _i([15, 6, -1], gpu), S2, None)
    # both are fp32 sums of the same terms in other orders: 2 x the bound of one of them, taken loosely
    # as (depth + 1) (d_k + 2 depth + 16) u = 1.7e-4 of sums whose terms are a few times their value
    for a, b in ((o, o2), (u, u2), (S, S2)):
        assert float((a - b).abs().max()) <= 4e-4 * float(a.abs().max())


def test_runs_twice_alike_and_side_by_side(gpu):
    """The same call again, and two calls on two streams at once, give the same bits."""
    kda = _kda()
    rng = np.random.default_rng(8)
    B, K, H = 16, 32, 8
    d, pool = _drafts(gpu, B, K, H, 128, 128, torch.bfloat16, 2 * B, 15)
    par = _i([sm.random_tree(rng, K, 6) for _ in range(B)], gpu)
    pages, outs = _i(list(range(B)), gpu), _i(list(range(B, 2 * B)), gpu)
    last = _i([random.Random(b).randint(-1, K - 1) for b in range(B)], gpu)

    def step(p):
        o, u = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], p, pages, par)
        return o, u, kda.kda_tree_commit(d["k"], d["alpha"], u, par, last, p, pages, outs)

    want = step(pool.clone())
    pools = [pool.clone() for _ in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s, p in zip(streams, pools):
        with torch.cuda.stream(s):
            got.append(step(p))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("where,value", [("v", float("nan")), ("v", float("inf")), ("v", 1e30), ("q", float("nan")), ("k", float("inf")),
                                         ("alpha", float("nan")), ("beta", float("inf"))])
@pytest.mark.parametrize("K", [14, 40])
def test_values_that_are_not_finite_stay_on_their_paths(gpu, where, value, K):
    """A drafted node whose values are not finite (or are huge) spoils the nodes that follow it, and no others:
    those keep the bounds."""
    kda = _kda()
    rng = np.random.default_rng(K)
    B, H, bad = 3, 2, 2
    d, pool = _drafts(gpu, B, K, H, 64, 64, torch.float32, 4, 40 + K)
    parents = [sm.random_tree(rng, K, 9) for _ in range(B)]
    d[where][1, bad, 1] = value
    o, u = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, _i([3, 0, 2], gpu), _i(parents, gpu))
    below = [t == bad for t in range(K)]
    for t in range(K):
        below[t] |= parents[1][t] >= 0 and below[parents[1][t]]
    assert 1 < sum(below) < K
    x, ho, hu, hp = {n: _host(t) for n, t in d.items()}, _host(o), _host(u), _host(pool)
    for b, page in enumerate([3, 0, 2]):
        for h in range(H):
            clean = [t for t in range(K) if not ((b, h) == (1, 1) and (t == bad if where == "q" else below[t]))]
            with np.errstate(all="ignore"):
                r = sm.tree_run(hp[page, h], *(x[n][b, :, h] for n in ("q", "k", "v", "alpha", "beta")), parents[b])
            sm.within(ho[b, clean, h], r["o"][clean], r["eo"][clean], sm.U, f"o of ({b}, {h})")
            sm.within(hu[b, h][clean], r["u"][clean], r["eu"][clean], sm.U, f"u of ({b}, {h})")
    if value != 1e30:  # and the node itself is not finite
        assert not np.isfinite(ho[1, bad, 1]).all()


def test_a_state_that_is_not_finite(gpu):
    """A NaN in one column of the state spoils that column of every node, and no other."""
    kda = _kda()
    K = 20
    d, pool = _drafts(gpu, 1, K, 1, 64, 128, torch.bfloat16, 1, 2)
    par = [sm.random_tree(np.random.default_rng(1), K, 5)]
    clean, _ = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, None, _i(par, gpu))
    pool[0, 0, 7, 33] = float("nan")
    o, _ = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, None, _i(par, gpu))
    assert torch.isnan(o[..., 33]).all()
    keep = torch.arange(128, device=gpu) != 33
    assert torch.isfinite(o[..., keep]).all()
    # (another order of the same sums: the bounds of both)
    x = {n: _host(t) for n, t in d.items()}
    pool[0, 0, 7, 33] = 0.0
    r = sm.tree_run(_host(pool)[0, 0], *(x[n][0, :, 0] for n in ("q", "k", "v", "alpha", "beta")), par[0])
    sm.within(_host(o)[0, :, 0][:, _host(keep).astype(bool)], r["o"][:, _host(keep).astype(bool)], r["eo"][:, _host(keep).astype(bool)], sm.U)
    sm.within(_host(clean)[0, :, 0][:, _host(keep).astype(bool)], r["o"][:, _host(keep).astype(bool)], r["eo"][:, _host(keep).astype(bool)], sm.U)


@pytest.mark.parametrize("K", [1, 9, 32, 64])
def test_captured_before_its_first_eager_call(gpu, K):
    """A shape whose first call is inside a capture, from another thread's stream, replayed on new trees."""
    import threading
    kda = _kda()
    rng = np.random.default_rng(K)
    B, H = 2, 3
    d, pool = _drafts(gpu, B, K, H, 32, 64, torch.float32, 3, K)
    par = _i([sm.random_tree(rng, K, 5) for _ in range(B)], gpu)
    o, u = torch.zeros(B, K, H, 64, device=gpu), torch.zeros(B, H, K, 64, device=gpu)
    graph = torch.cuda.CUDAGraph()

    def capture():
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, None, par, o=o, u=u)

    torch.cuda.synchronize()
    t = threading.Thread(target=capture)
    t.start()
    t.join()
    for _ in range(3):
        par.copy_(_i([sm.random_tree(rng, K, 5) for _ in range(B)], gpu))
        d["q"].mul_(1.25)
        graph.replay()
        wo, wu = kda.kda_tree_verify(d["q"], d["k"], d["v"], d["alpha"], d["beta"], pool, None, par)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(u, wu)
