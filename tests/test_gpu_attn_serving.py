"""The calls of an attention layer together, as a server of a hybrid model would run them, against the definitions in 64
bits: prompts turned, cached and attended to, a sample forked off, drafts appended and verified, a token decoded, a next turn
behind the cached prefix, a sequence ended and the pool packed; then a step beside a recurrent layer's, replayed from a graph."""
import pytest
import torch

import attention_model as am
import kda_inputs as ki

pytestmark = pytest.mark.gpu
BF, E = torch.bfloat16, torch.float8_e4m3fn


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _cu(lens, gpu):
    return _i([sum(lens[:i]) for i in range(len(lens) + 1)], gpu)


def _decoded(q, lay, pool, table, rows, lens):
    """(o, slack) of the definition on what the pages hold."""
    m, t = am.Pages(lay, pool), table.tolist()
    B, K, Hq, _ = q.shape
    for b in range(B):
        k, v, _ = m.tokens(t[rows[b]], lens[b])
        seen = torch.arange(K) + lens[b] - K + 1
        yield [torch.stack(x, 1) for x in zip(*(am.attend(q[b, :, h].cpu(), k[:, h * lay.H // Hq], v[:, h * lay.H // Hq], seen, lay.d_k ** -0.5, am.HALF[BF])
                                                for h in range(Hq)))]


@pytest.mark.parametrize("dtype", [BF, E])
def test_a_turn_of_a_server(gpu, dtype):
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(1)
    lay = kda.KVLayout(dtype, 16, 2, 64, 64)
    Hq, L, P, W = 6, 2, 24, 8
    freq = 10000.0 ** (-torch.arange(32, device=gpu).float() / 32)
    pools = torch.randint(0, 120, (L, P, lay.page_bytes), generator=g, device=gpu, dtype=torch.uint8)  # (anything on the free pages)
    table, ref = torch.full((4, W), -1, dtype=torch.int32, device=gpu), torch.zeros(P, dtype=torch.int32, device=gpu)

    def tokens(n):
        row = torch.randn(n, Hq + 4, 64, generator=g, device=gpu).to(BF)  # a fused projection's
        return row[:, :Hq], row[:, Hq:Hq + 2], row[:, Hq + 2:]

    # two prompts on three pages each, on every layer
    kda.kda_cache_fork(table, ref, _i([-1, -1], gpu), _i([0, 1], gpu), 3)
    lens = [40, 33]
    for pool in pools:
        q, k, v = tokens(73)
        kt = torch.empty(73, 2, 64, device=gpu, dtype=BF)
        qt, _ = kda.kda_kv_append(k, v, pool, lay, table, _i([0, 0], gpu), cu_seqlens=_cu(lens, gpu), q=q, inv_freq=freq, k_out=kt)
        pos = list(range(40)) + list(range(33))
        am.close(qt, *am.turn(q.cpu(), pos, freq, "halves"))
        am.close(kt, *am.turn(k.cpu(), pos, freq, "halves"))
        o = kda.kda_attn_fwd(qt, kt, v, cu_seqlens=_cu(lens, gpu))
        am.close(o, *am.fwd(qt, kt, v, 0.125, lens))
        # a prompt's last row is what decoding its last token gives, as far as the pages' rounding goes (bf16: to bf16's)
        last = kda.kda_attn_decode(qt[[39, 72]].contiguous(), pool, lay, table, _i(lens, gpu), rows=_i([0, 1], gpu))
        for b, want in enumerate(_decoded(qt[[39, 72]][:, None], lay, pool, table, [0, 1], lens)):
            am.close(last[b:b + 1], *want)
        if dtype == BF:
            assert float((last.float() - o[[39, 72]].float()).abs().max()) < 0.05
    # the first is answered twice: whole pages shared, the page that is still filling copied
    kda.kda_cache_fork(table, ref, _i([0], gpu), _i([2], gpu), 0)
    own, free = table[2, 2].item(), (ref == 0).nonzero()[0].item()
    kda.kda_cache_copy(pools, _i([[own, free]], gpu), n_layers=L)
    table[2, 2] = free
    ref[free] += 1
    ref[own] -= 1
    rows, lens = [0, 2, 1], [40, 40, 33]
    for pool in pools:
        # four drafted tokens each
        q, k, v = tokens(12)
        before = pool.clone()
        qt, _ = kda.kda_kv_append(k, v, pool, lay, table, _i(lens, gpu), rows=_i(rows, gpu), cu_seqlens=_cu([4, 4, 4], gpu), q=q, inv_freq=freq)
        assert torch.equal(pool[table[0, :2].long()], before[table[0, :2].long()]), "shared pages"
        o = kda.kda_attn_decode(qt.unflatten(0, (3, 4)), pool, lay, table, _i([44, 44, 37], gpu), rows=_i(rows, gpu))
        for b, want in enumerate(_decoded(qt.unflatten(0, (3, 4)), lay, pool, table, rows, [44, 44, 37])):
            am.close(o[b], *want, what=f"drafts of row {rows[b]}")
        # two, none and all of them accepted; one more token each
        lens1 = [42, 40, 37]
        q, k, v = tokens(3)
        qt, _ = kda.kda_kv_append(k, v, pool, lay, table, _i(lens1, gpu), rows=_i(rows, gpu), q=q, inv_freq=freq)
        o = kda.kda_attn_decode(qt, pool, lay, table, _i([n + 1 for n in lens1], gpu), rows=_i(rows, gpu))
        for b, want in enumerate(_decoded(qt[:, None], lay, pool, table, rows, [n + 1 for n in lens1])):
            am.close(o[b:b + 1], *want, what=f"token of row {rows[b]}")
        # the next turn of rows 0 and 2: 5 and 3 new tokens behind the cached ones
        n, m = [5, 3], [43, 41]
        q, k, v = tokens(8)
        kt = torch.empty(8, 2, 64, device=gpu, dtype=BF)
        qt, _ = kda.kda_kv_append(k, v, pool, lay, table, _i(m, gpu), rows=_i([0, 2], gpu), cu_seqlens=_cu(n, gpu), q=q, inv_freq=freq, k_out=kt)
        kc, vc = kda.kda_kv_read(pool, lay, table, _cu(m, gpu), sum(m), rows=_i([0, 2], gpu))
        ks, vs = torch.cat([kc[:43], kt[:5], kc[43:], kt[5:]]), torch.cat([vc[:43], v[:5], vc[43:], v[5:]])
        both = [48, 44]
        o = kda.kda_attn_fwd(qt, ks, vs, cu_seqlens=_cu(n, gpu), cu_seqlens_k=_cu(both, gpu))
        am.close(o, *am.fwd(qt, ks, vs, 0.125, n, both))
    # the second prompt ends; the pool is packed, and answers as before
    q = torch.randn(2, Hq, 64, generator=g, device=gpu).to(BF)
    want = [kda.kda_attn_decode(q, pool, lay, table, _i([48, 44], gpu), rows=_i([0, 2], gpu)) for pool in pools]
    kda.kda_cache_free(table, ref, _i([1], gpu))
    t2, r2, moves, n, live = kda.kda_cache_compact(table, ref)
    kda.kda_cache_copy(pools, moves, n, n_layers=L)
    assert int(live) == 4 and int(t2.max()) == 3
    for pool, w in zip(pools, want):
        assert torch.equal(kda.kda_attn_decode(q, pool, lay, t2, _i([48, 44], gpu), rows=_i([0, 2], gpu)), w)


@pytest.mark.parametrize("width", [6, 300])
def test_a_step_beside_a_recurrent_layer_replayed(gpu, width):
    """One graph with a recurrent layer's decode and an attention layer's append and decode, replayed as the sequences grow;
    every replay equals the eager calls."""
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(2)
    B, H, d = 3, 4, 64
    lay = kda.KVLayout(E, 16, 2, d, d)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, :6] = torch.randperm(18, generator=torch.Generator().manual_seed(3)).view(3, 6).to(torch.int32)
    table = table.to(gpu)
    tok = ki.make_decode_token(B, H, d, d, BF, seed=4, device=gpu)
    freq = 10000.0 ** (-torch.arange(32, device=gpu).float() / 32)
    q, k, v = (torch.randn(B, h, d, generator=g, device=gpu).to(BF) for h in (8, 2, 2))
    lens, rows, state_pages = _i([0, 20, 47], gpu), _i([0, 1, 2], gpu), _i([2, 0, 1], gpu)
    need = kda.kda_attn_decode_plan(lay, B, 1, 8, width)

    def made():
        return dict(pool=lay.pool(18, gpu), states=ki.make_state(4, H, d, d, 0.1, 5, gpu), qo=torch.zeros_like(q), o=torch.zeros_like(q),
                    os=torch.zeros(B, H, d, device=gpu), seen=torch.zeros_like(lens), ws=torch.empty(max(need, 16), dtype=torch.uint8, device=gpu))

    def step(x):
        kda.kda_decode_step_paged(*(tok[n] for n in ("q", "k", "v", "alpha", "beta")), x["states"], state_pages, o=x["os"])
        kda.kda_kv_append(k, v, x["pool"], lay, table, lens, rows=rows, q=q, inv_freq=freq, q_out=x["qo"])
        torch.add(lens, 1, out=x["seen"])
        kda.kda_attn_decode(x["qo"], x["pool"], lay, table, x["seen"], rows=rows, o=x["o"], workspace=x["ws"])

    a, b = made(), made()
    step(made())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(20):
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(a[n], b[n]) for n in a if n != "ws"), f"replay {i}"
        lens += 1
        for x in (q, k, v, tok["q"]):
            x.copy_(torch.randn(x.shape, generator=g, device=gpu).to(BF))
        if i == 9:
            rows.copy_(_i([0, -1, 2], gpu))  # one sequence ends
    for c, want in enumerate(_decoded(a["qo"][:, None], lay, a["pool"], table, [0, 1, 2], a["seen"].tolist())):
        if c != 1:
            am.close(a["o"][c:c + 1], *want)
