"""The serving operators together, as a server would run them, against the recurrence in 64 bits: projections
normalised, prompts prefilled into pages, samples forked, a tree of drafts verified and committed, one more token
decoded, a sample ended and the pool packed; then the tree step and the decode replayed from a graph."""
import numpy as np
import pytest
import torch

import serving_model as sm

pytestmark = pytest.mark.gpu


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _tokens(kda, gpu, g, lead, H, dk, dv):
    """Normalised tokens [*lead][H] from the rows of a fused projection."""
    rows = torch.randn(*lead, H, 2 * dk + dv, generator=g, device=gpu)
    q, k = rows[..., :dk].contiguous(), rows[..., dk:2 * dk].contiguous()
    kda.kda_qk_norm(q.reshape(-1, H, dk), k.reshape(-1, H, dk), q_scale=dk ** -0.5, q_out=q.view(-1, H, dk), k_out=k.view(-1, H, dk))
    return dict(q=q, k=k, v=rows[..., 2 * dk:].contiguous(),
                alpha=torch.sigmoid(torch.randn(*lead, H, dk, generator=g, device=gpu) + 3),
                beta=torch.sigmoid(torch.randn(*lead, H, generator=g, device=gpu)))


def _after(S, tok, b, path):
    """The states [H][dk][dv] (float64) of S after tokens path of tok[b], and the last token's outputs [H][dv]."""
    x = {n: t[b].double().cpu().numpy() for n, t in tok.items()}
    S, o = S.copy(), np.zeros((S.shape[0], S.shape[2]))
    for h in range(S.shape[0]):
        for t in path:
            Sb = x["alpha"][t, h][:, None] * S[h]
            S[h] = Sb + np.outer(x["k"][t, h], x["beta"][t, h] * (x["v"][t, h] - Sb.T @ x["k"][t, h]))
        o[h] = S[h].T @ x["q"][path[-1], h]
    return S, o


def test_a_turn_of_a_server(gpu):
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(1)
    L, P, H, dk, dv, T = 2, 12, 3, 64, 64, 40
    pools = torch.randn(L, P, H, dk, dv, generator=g, device=gpu)  # (garbage on the free pages)
    table, ref = torch.full((6, 2), -1, dtype=torch.int32, device=gpu), torch.zeros(P, dtype=torch.int32, device=gpu)
    # two prompts start on zeroed pages and are prefilled on every layer
    moves, n = kda.kda_cache_fork(table, ref, _i([-1, -1], gpu), _i([2, 4], gpu))
    kda.kda_cache_copy(pools, moves, n, n_layers=L)
    assert table[[2, 4], 0].tolist() == [0, 1] and int(n) == 2 and not pools[:, :2].any()
    prompts = [_tokens(kda, gpu, g, (2, T), H, dk, dv) for _ in range(L)]
    ref_states = {}
    for layer in range(L):
        x = prompts[layer]
        assert float((x["k"].norm(dim=-1) - 1).abs().max()) < 1e-5
        _, S = kda.kda_chunk_fwd(x["q"], x["k"], x["v"], x["alpha"], x["beta"], pools[layer, :2].contiguous(), chunk=32)
        kda.kda_cache_copy(pools[layer], _i([[0, 0], [1, 1]], gpu), src=S)
        for b in range(2):
            ref_states[layer, b], _ = _after(np.zeros((H, dk, dv)), x, b, range(T))
    # the first prompt is answered three times
    moves, n = kda.kda_cache_fork(table, ref, _i([2, 2], gpu), _i([0, 5], gpu))
    kda.kda_cache_copy(pools, moves, n, n_layers=L)
    rows = [2, 4, 0, 5]
    pages = table[rows, 0].contiguous()
    assert pages.tolist() == [0, 1, 2, 3]
    par = [[-1, 0, 0, 1, -1], [-1, 0, 1, 2, 3], [-1, -1, -1, -1, -1], [-1, 0, 0, 2, 2]]
    paths = {0: [0, 1, 3], 1: [0, 1, 2, 3, 4], 2: [], 3: [0, 2, 4]}
    last = _i([3, 4, -1, 4], gpu)
    for layer in range(L):
        x = _tokens(kda, gpu, g, (4, 5), H, dk, dv)
        o, u = kda.kda_tree_verify(x["q"], x["k"], x["v"], x["alpha"], x["beta"], pools[layer], pages, _i(par, gpu))
        kda.kda_tree_commit(x["k"], x["alpha"], u, _i(par, gpu), last, pools[layer], pages)
        y = _tokens(kda, gpu, g, (4, 1), H, dk, dv)
        od = kda.kda_decode_step_paged(*(y[m][:, 0].contiguous() for m in ("q", "k", "v", "alpha", "beta")), pools[layer], pages)
        for b in range(4):
            S = ref_states[layer, 0 if b != 1 else 1]
            if paths[b]:
                S, want = _after(S, x, b, paths[b])
                assert np.abs(o[b, paths[b][-1]].cpu().numpy() - want).max() < 2e-4
            S, want = _after(S, y, b, [0])
            ref_states[layer, "row", b] = S
            # (fp32 over 46 tokens of values near 1: the oracle's own fp32 tolerance is 1e-4 for T = 64)
            assert np.abs(od[b].cpu().numpy() - want).max() < 2e-4
    # a sample ends; the pool is packed
    kda.kda_cache_free(table, ref, _i([4], gpu))
    t2, r2, moves, n, live = kda.kda_cache_compact(table, ref)
    kda.kda_cache_copy(pools, moves, n, n_layers=L)
    assert int(live) == 3 and t2[[2, 4, 0, 5], 0].tolist() == [0, -1, 2, 1] and r2.tolist() == [1, 1, 1] + [0] * (P - 3)
    for layer in range(L):
        for b, page in ((0, 0), (2, 2), (3, 1)):
            assert np.abs(pools[layer, page].cpu().numpy() - ref_states[layer, "row", b]).max() < 2e-4


@pytest.mark.parametrize("K", [24, 64])
def test_tree_step_and_decode_replayed(gpu, K):
    """One graph with a tree step (the largest takes more LDS than a launch has by default) and a decode; every
    replay equals the eager calls on the same lists."""
    kda = _kda()
    B, H, dk, dv, P = 4, 4, 128, 128, 9
    rng = np.random.default_rng(2)
    g = torch.Generator(device=gpu).manual_seed(3)
    x, y = _tokens(kda, gpu, g, (B, K), H, dk, dv), _tokens(kda, gpu, g, (B, 1), H, dk, dv)
    y = {n: t[:, 0].contiguous() for n, t in y.items()}
    pool = 0.1 * torch.randn(P, H, dk, dv, generator=g, device=gpu)
    pages, par, nodes, last = _i([0, 3, 5, -1], gpu), _i([sm.random_tree(rng, K, 6)] * B, gpu), _i([K] * B, gpu), _i([3] * B, gpu)
    o, u, od = torch.zeros(B, K, H, dv, device=gpu), torch.zeros(B, H, K, dv, device=gpu), torch.zeros(B, H, dv, device=gpu)

    def step(pool, o, u, od):
        kda.kda_tree_verify(x["q"], x["k"], x["v"], x["alpha"], x["beta"], pool, pages, par, nodes, o=o, u=u)
        kda.kda_tree_commit(x["k"], x["alpha"], u, par, last, pool, pages, None, nodes)
        kda.kda_decode_step_paged(y["q"], y["k"], y["v"], y["alpha"], y["beta"], pool, pages, o=od)

    other = [t.clone() for t in (pool, o, u, od)]
    step(*[t.clone() for t in other])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, o, u, od)
    for i in range(4):
        par.copy_(_i([sm.random_tree(rng, K, 6) for _ in range(B)], gpu))
        nodes.copy_(_i([K - i, K, 5, 3], gpu)), last.copy_(_i([i, -1, 4, 2], gpu)), pages.copy_(_i([i, 4, 8, -1], gpu))
        graph.replay()
        step(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((pool, o, u, od), other))


@pytest.mark.parametrize("helper", [True, False])
def test_binding_refuses_what_does_not_fit(gpu, helper, monkeypatch):
    """Shapes, types, strides and devices that do not fit raise before the library is called, with the compiled
    argument helper and without it; calls that fit give the same results both ways."""
    kda = _kda()
    if helper:
        assert kda._need is not kda._need_in_words, "the argument helper is not built"
    else:
        monkeypatch.setattr(kda, "_need", kda._need_in_words)
        monkeypatch.setattr(kda, "_rows", lambda t, dtype, index: None)
    f = lambda *s, dtype=torch.float32: torch.randn(*s, device=gpu).to(dtype)  # noqa: E731
    q, bf = f(6, 4, 32), f(6, 4, 32, dtype=torch.bfloat16)
    for bad in (dict(q=q[:, :, ::2]), dict(q=q[:, ::2]), dict(q=q[0]), dict(q=q.double()), dict(q=q, k=bf), dict(q=q, k=q[:5]),
                dict(q=q, k=f(6, 4, 16)), dict(q=q, k=q.cpu()), dict(q=q, norm="l1"), dict(q=q, pairing=0),
                dict(q=q, q_weight=f(31)), dict(q=q, inv_freq=f(8)), dict(q=q, inv_freq=f(8), positions=_i([1, 2], gpu)),
                dict(q=q, q_out=f(6, 4, 16)), dict(q=q, q_out=bf, out_dtype=torch.float32), dict(q=q, out_dtype=torch.float16),
                dict(q=f(3, 4, 2, 32)[:, ::2].transpose(0, 1), k=None), dict(q=q, k_out=q)):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_qk_norm(**bad)
    with pytest.raises(kda.KdaError, match="ALIAS"):
        kda.kda_qk_norm(q, q.clone(), k_out=q)
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        kda.kda_qk_norm(f(2, 2, 20))
    table, ref, one = _i([[0, 1], [-1, -1]], gpu), _i([1, 1, 0], gpu), _i([1], gpu)
    for call in (lambda: kda.kda_cache_fork(table, ref, one, _i([0, 1], gpu)), lambda: kda.kda_cache_fork(table.t(), ref, one, one),
                 lambda: kda.kda_cache_fork(table, ref.float(), one, one), lambda: kda.kda_cache_fork(table, ref, one, one, 2, moves=_i([[0, 0]], gpu)),
                 lambda: kda.kda_cache_free(table, ref, one.long()), lambda: kda.kda_cache_free(table[0], ref, one),
                 lambda: kda.kda_cache_compact(table, ref, table_out=table[:1]), lambda: kda.kda_cache_compact(table, ref, moves=one),
                 lambda: kda.kda_cache_copy(q, _i([0, 1], gpu)), lambda: kda.kda_cache_copy(q, _i([[0, 1]], gpu), src=bf),
                 lambda: kda.kda_cache_copy(q, _i([[0, 1]], gpu), n_layers=3), lambda: kda.kda_cache_copy(q, _i([[0, 1]], gpu), src=f(6, 4, 16))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(kda.KdaError, match="SHAPE"):
        kda.kda_cache_fork(table, ref, one, one, 3)
    assert table.tolist() == [[0, 1], [-1, -1]] and ref.tolist() == [1, 1, 0]
    # calls that fit
    y, _ = kda.kda_qk_norm(q.reshape(2, 3, 4, 32))
    assert torch.allclose(y.reshape(6, 4, 32), q / q.norm(dim=-1, keepdim=True), atol=1e-5)
    moves, n = kda.kda_cache_fork(table, ref, _i([0], gpu), one)
    assert table.tolist() == [[0, 1], [2, 1]] and ref.tolist() == [1, 2, 1] and int(n) == 1
    pool = f(3, 2, 16, 16)
    kda.kda_cache_copy(pool, moves, n)
    tok = {m: f(1, 2, 16) for m in ("q", "k", "v")}
    o = kda.kda_decode_step_paged(tok["q"], tok["k"], tok["v"], torch.full((1, 2, 16), 0.5, device=gpu), f(1, 2), pool, _i([2], gpu))
    assert torch.isfinite(o).all() and not torch.equal(pool[2], pool[0])
    with pytest.raises((ValueError, TypeError)):
        kda.kda_decode_step_paged(tok["q"], tok["k"], tok["v"], None, f(1, 2), pool, _i([2], gpu))
    with pytest.raises((ValueError, TypeError)):
        kda.kda_tree_verify(tok["q"], tok["k"], tok["v"], tok["q"], f(1, 2), pool, None, one)


def test_head_norms_feed_the_recurrence(gpu):
    """Keys as a fused projection leaves them, normalised in place and prefilled: the oracle on the same keys."""
    import kda_inputs as ki
    from kda_check import assert_close, gpu_o_heads, gpu_s_heads, oracle_prefill
    kda = _kda()
    B, T, H, d = 2, 130, 3, 64
    x = ki.make_prefill(B, T, H, d, d, torch.bfloat16, 3.0, 0.1, seed=5, device=gpu)
    rows = torch.randn(B, T, 3 * H, d, device=gpu).to(torch.bfloat16)
    q, k = rows[:, :, :H], rows[:, :, H:2 * H]
    x["q"], x["k"] = kda.kda_qk_norm(q, k, q_scale=d ** -0.5)
    x["v"] = rows[:, :, 2 * H:].contiguous()
    o, S = kda.kda_chunk_fwd(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S0"])
    torch.cuda.synchronize()
    ro, rs = oracle_prefill(x)
    assert_close(gpu_o_heads(o), ro, True, "o")
    assert_close(gpu_s_heads(S), rs, True, "S_T")
