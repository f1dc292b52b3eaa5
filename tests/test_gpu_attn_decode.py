"""kda_attn_decode against the definition in 64 bits: types, head sizes, groups, drafted tokens, page sizes, lengths from
nothing to long ones, pages out of range, what the pages hold behind a sequence, shared workspaces, graphs."""
import math

import pytest
import torch

import attention_model as am

pytestmark = pytest.mark.gpu
BF, F, E = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _pool(lay, P, gpu, seed, spoil=True):
    """A pool of finite codes and scales."""
    g = torch.Generator(device=gpu).manual_seed(seed)
    pool = lay.pool(P, gpu)
    k, v, s = lay.views(pool)
    for x in (k, v):
        x.copy_(torch.randn(x.shape, generator=g, device=gpu).mul_(20 if lay.dtype == E else 1).to(x.dtype))
    if s is not None:
        s.copy_(torch.exp2(torch.randint(-6, -3, s.shape, generator=g, device=gpu).float()))
    return pool


def _spoil(lay, pool, table, rows, lens, bad=math.nan):
    """Everything that no sequence holds becomes `bad`: the free pages, and the places behind each sequence's last token."""
    k, v, s = lay.views(pool)
    keep = torch.zeros(pool.shape[0], lay.page_tokens, dtype=torch.bool)
    for r, n in zip(rows, lens):
        for t in range(min(max(n, 0), lay.page_tokens * len(table[0]))):
            j = t // lay.page_tokens
            if 0 <= r < len(table) and j < len(table[r]) and 0 <= table[r][j] < len(keep):
                keep[table[r][j], t % lay.page_tokens] = True
    keep = keep.to(pool.device)
    for x in (k, v):
        x.copy_(torch.where(keep[:, None, :, None], x.float(), bad).to(x.dtype))
    if s is not None:
        s.copy_(torch.where(keep.any(1)[:, None, None], s, bad))


def _table(need, gpu, seed, width=None, extra=3):
    P = sum(need) + extra
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    t = torch.full((len(need), width or max(max(need), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b + 1])], dtype=torch.int32)
    return P, t


def _model(q, lay, pool, table, rows, lens, scale):
    """(o, slack) for q [B][K][Hq][dk]; padding: None."""
    m, out = am.Pages(lay, pool), []
    B, K, Hq, _ = q.shape
    G = Hq // lay.H
    p_half = am.HALF[BF] if q.dtype == BF else 0.0
    for b in range(B):
        if not 0 <= rows[b] < len(table):
            out.append(None)
            continue
        n = min(max(lens[b], 0), len(table[0]) * lay.page_tokens)
        k, v, there = m.tokens(table[rows[b]], n)
        seen = torch.tensor([int(there[:max(n - K + 1 + t, 0)].sum()) for t in range(K)])  # (of those that are there)
        o, sl = torch.zeros(K, Hq, lay.d_v, dtype=torch.float64), torch.zeros(K, Hq, lay.d_v, dtype=torch.float64)
        for h in range(Hq):
            o[:, h], sl[:, h] = am.attend(q[b, :, h].cpu(), k[there, h // G], v[there, h // G], seen, scale, p_half)
        out.append((o, sl))
    return out


def _check(gpu, lay, lens, K=1, hq=None, dtype=BF, o_dtype=None, rows=None, table=None, P=None, width=None, seed=1, scale=None, q=None, bad=math.nan):
    kda = _kda()
    B = len(lens)
    if table is None:
        P, table = _table([-(-max(n, 0) // lay.page_tokens) for n in lens], gpu, seed, width)
        table = table.tolist()
    rows = list(range(B)) if rows is None else rows
    pool = _pool(lay, P, gpu, seed + 1)
    if bad is not None:
        _spoil(lay, pool, table, rows, lens, bad)
    hq = hq or 2 * lay.H
    if q is None:
        q = torch.randn(B, K, hq, lay.d_k, generator=torch.Generator(device=gpu).manual_seed(seed + 2), device=gpu).to(dtype)
    o = torch.full((B, K, hq, lay.d_v), 7.0, device=gpu, dtype=o_dtype or dtype)
    kda.kda_attn_decode(q, pool, lay, _i(table, gpu), _i(lens, gpu), rows=_i(rows, gpu), o=o, scale=scale)
    torch.cuda.synchronize()
    for b, want in enumerate(_model(q, lay, pool, table, rows, lens, lay.d_k ** -0.5 if scale is None else scale)):
        if want is None:
            assert bool((o[b] == 7).all()), "padding"
        else:
            am.close(o[b], *want, what=f"sequence {b} of {lens[b]}")
    return o


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("width", [None, 200])
def test_types_and_head_sizes(gpu, dtype, cache, dk, dv, width):
    """Both forms: units taken whole (short rows), and shared out (long rows)."""
    lay = _kda().KVLayout(cache, 32, 2, dk, dv)
    _check(gpu, lay, [1, 33, 300, 1000], dtype=dtype, o_dtype=F, width=width)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("pt", [16, 32, 64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_lengths_and_pages(gpu, cache, pt, wide):
    lay = _kda().KVLayout(cache, pt, 1, 64, 64)
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 255, 256, 257, 500, 513, -3]
    o = _check(gpu, lay, lens, width=4096 // pt if wide else None)
    assert not o[0].any() and not o[-1].any()


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("hq,hk,K", [(1, 1, 1), (8, 8, 1), (5, 1, 1), (16, 1, 1), (17, 1, 1), (40, 2, 1), (8, 2, 4), (8, 8, 5), (12, 2, 16), (40, 8, 3)])
@pytest.mark.parametrize("wide", [False, True])
def test_groups_and_drafts(gpu, cache, hq, hk, K, wide):
    lay = _kda().KVLayout(cache, 16, hk, 64, 64)
    _check(gpu, lay, [K, K + 1, 100, 260, K - 1, 1], K=K, hq=hq, width=300 if wide else None)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("dtype", [BF, F])
def test_long(gpu, cache, dtype):
    """A long sequence that many workgroups share beside short ones."""
    lay = _kda().KVLayout(cache, 64, 2, 128, 128)
    _check(gpu, lay, [70001, 3, 0, 5000, 129], dtype=dtype, o_dtype=F)


@pytest.mark.parametrize("n", [2049, 8193, 32767, 65537, 75393, 140001])
def test_units_that_many_workgroups_share(gpu, n):
    """One head: up to 512 parts to join."""
    kda = _kda()
    _check(gpu, kda.KVLayout(E, 128, 1, 64, 64), [n], K=2, hq=2, seed=40)


@pytest.mark.parametrize("wide", [False, True])
def test_padding_and_rows(gpu, wide):
    lay = _kda().KVLayout(E, 16, 2, 64, 64)
    need = [3, 5, 1, 9]
    P, table = _table(need, gpu, 5, 200 if wide else None)
    _check(gpu, lay, [140, 10, 77, 3, 50, 40], rows=[3, 2, 1, -1, 4, 0], table=table.tolist(), P=P)


@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("wide", [False, True])
def test_pages_out_of_range_are_not_seen(gpu, K, cache, wide):
    lay = _kda().KVLayout(cache, 16, 2, 64, 64)
    w = 200 if wide else 6
    table = [[0, -1, 2, 99, 4, 5], [-1] * 6, [7, 8, 9, -5, 2 ** 31 - 1, 10], [11, 12, -1, -1, -1, -1]]
    _check(gpu, lay, [96, 96, 50, 40], K=K, table=[r + [-1] * (w - 6) for r in table], P=13)


@pytest.mark.parametrize("wide", [False, True])
def test_lengths_behind_the_row(gpu, wide):
    """A length past the row's end is cut to it."""
    lay = _kda().KVLayout(BF, 16, 1, 64, 64)
    P, table = _table([2, 3], gpu, 6, 150 if wide else 3)
    _check(gpu, lay, [2 ** 31 - 1, 1000], table=table.tolist(), P=P)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, 3e38, None])
@pytest.mark.parametrize("cache", [BF, E])
def test_what_lies_behind_a_sequence_has_no_influence(gpu, cache, bad):
    lay = _kda().KVLayout(cache, 64, 2, 64, 64)
    for K in (1, 3):
        _check(gpu, lay, [5, 64, 70, 130], K=K, bad=bad)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_bad_draft_has_no_influence_on_earlier_tokens(gpu, cache, wide, dtype):
    """Keys or values of a drafted token that are not finite: the tokens before it are what they were, it and the later ones not finite."""
    kda = _kda()
    lay = kda.KVLayout(cache, 16, 2, 64, 64)
    lens, K = [35, 100, 16], 4
    P, table = _table([-(-n // 16) for n in lens], gpu, 7, 300 if wide else None)
    table = table.to(gpu)
    pool = _pool(lay, P, gpu, 8)
    q = torch.randn(3, K, 4, 64, generator=torch.Generator(device=gpu).manual_seed(9), device=gpu).to(dtype)
    clean = kda.kda_attn_decode(q, pool, lay, table, _i(lens, gpu), o_dtype=F)
    ref = _model(q, lay, pool, table.tolist(), [0, 1, 2], lens, 0.125)
    for which in (0, 1):
        for t in range(K):
            p2 = pool.clone()
            x = lay.views(p2)[which]
            for b, n in enumerate(lens):
                at = n - K + t
                x[int(table[b, at // 16]), 1, at % 16] = math.nan
            o = kda.kda_attn_decode(q, p2, lay, table, _i(lens, gpu), o_dtype=F)
            assert torch.equal(o[:, :, :2], clean[:, :, :2]), "another head"
            for b in range(3):
                am.close(o[b, :t], ref[b][0][:t], ref[b][1][:t], f"sequence {b}, before draft {t}")
            assert torch.isnan(o[:, t:, 2:]).all()


def test_scales_of_all_sizes(gpu):
    """Pages whose scales differ by powers of two, zeros among them."""
    kda = _kda()
    lay = kda.KVLayout(E, 16, 1, 64, 64)
    P, table = _table([20], gpu, 10)
    pool = _pool(lay, P, gpu, 11)
    s = lay.views(pool)[2]
    s.copy_(torch.exp2(torch.arange(s.numel(), device=gpu).view(s.shape).float() % 23 - 18))
    s[3] = 0.0
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator(device=gpu).manual_seed(12), device=gpu)
    for dt in (BF, F):
        o = kda.kda_attn_decode(q.to(dt), pool, lay, table.to(gpu), _i([310], gpu), o_dtype=F)
        am.close(o[0], *_model(q.to(dt), lay, pool, table.tolist(), [0], [310], 0.125)[0])


def test_many_sequences(gpu):
    """As many sequences as a call takes, lengths of all sizes, most of them padding or empty."""
    kda = _kda()
    lay = kda.KVLayout(BF, 16, 1, 64, 64)
    B = 4096
    lens = [0] * B
    for b, n in ((0, 5), (1, 3000), (700, 17), (2048, 1), (4000, 900), (4095, 64)):
        lens[b] = n
    need = [-(-n // 16) for n in lens]
    P, table = _table(need, gpu, 13)
    pool = _pool(lay, P, gpu, 14)
    rows = [b if b % 3 or lens[b] else -1 for b in range(B)]
    q = torch.randn(B, 2, 64, generator=torch.Generator(device=gpu).manual_seed(15), device=gpu).to(BF)
    o = kda.kda_attn_decode(q, pool, lay, table.to(gpu), _i(lens, gpu), rows=_i(rows, gpu))
    some = [b for b in range(B) if lens[b]]
    ref = _model(q[some][:, None], lay, pool, table.tolist(), some, [lens[b] for b in some], 0.125)
    for b, want in zip(some, ref):
        am.close(o[b:b + 1], *want, what=f"sequence {b}")
    rest = torch.ones(B, dtype=torch.bool, device=gpu)
    rest[some] = False
    assert not o[rest].any()


def test_far_pages(gpu):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    kda = _kda()
    for dt in (E, BF):
        lay = kda.KVLayout(dt, 128, 64, 128, 128)
        P = 2100 if dt == E else 1100
        pool = torch.empty(P, lay.page_bytes, dtype=torch.uint8, device=gpu)
        small = _pool(lay, 3, gpu, 16)
        assert (P - 3) * lay.page_bytes > 2 ** 32
        pool[P - 3:] = small
        q = torch.randn(1, 64, 128, device=gpu).to(BF)
        o = kda.kda_attn_decode(q, pool, lay, _i([[P - 1, P - 3, P - 2]], gpu), _i([300], gpu))
        assert torch.equal(o, kda.kda_attn_decode(q, small, lay, _i([[2, 0, 1]], gpu), _i([300], gpu)))


def test_workspaces(gpu):
    """A given workspace whatever it holds; runs are bit-equal; two streams with a workspace each."""
    kda = _kda()
    lay = kda.KVLayout(E, 64, 2, 128, 128)
    lens = [9000, 100, 4000]
    P, table = _table([-(-n // 64) for n in lens], gpu, 17)
    pool, table = _pool(lay, P, gpu, 18), table.to(gpu)
    q = torch.randn(3, 8, 128, generator=torch.Generator(device=gpu).manual_seed(19), device=gpu).to(BF)
    need = kda.kda_attn_decode_plan(lay, 3, 1, 8, table.shape[1])
    want = kda.kda_attn_decode(q, pool, lay, table, _i(lens, gpu))
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=gpu)
        assert torch.equal(kda.kda_attn_decode(q, pool, lay, table, _i(lens, gpu), workspace=ws), want)
    with pytest.raises(kda.KdaError, match="SHAPE"):
        kda.kda_attn_decode(q, pool, lay, table, _i(lens, gpu), workspace=ws[:-16])
    ln = _i(lens, gpu)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        outs += [kda.kda_attn_decode(q, pool, lay, table, ln, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("wide", [False, True])
def test_captured(gpu, wide):
    kda = _kda()
    lay = kda.KVLayout(E, 16, 2, 64, 64)
    P, table = _table([20, 20, 20], gpu, 20, 400 if wide else None)
    pool, table = _pool(lay, P, gpu, 21), table.to(gpu)
    q = torch.randn(3, 2, 8, 64, generator=torch.Generator(device=gpu).manual_seed(22), device=gpu).to(BF)
    lens, rows = _i([1, 2, 3], gpu), _i([0, 1, 2], gpu)
    o = torch.zeros(3, 2, 8, 64, device=gpu, dtype=BF)
    kda.kda_attn_decode(q, pool, lay, table, lens, rows=rows, o=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_attn_decode(q, pool, lay, table, lens, rows=rows, o=o)
    for ln, r in (([300, 2, 40], [0, 1, 2]), ([5, 310, 0], [2, -1, 0]), ([320, 320, 320], [1, 1, 1]), ([17, 1, 200], [-1, 0, 1])):
        lens.copy_(_i(ln, gpu)), rows.copy_(_i(r, gpu)), q.mul_(-1), o.fill_(7)
        graph.replay()
        want = torch.full_like(o, 7.0)
        kda.kda_attn_decode(q, pool, lay, table, lens, rows=rows, o=want)
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_binding_refusals(gpu):
    kda = _kda()
    lay = kda.KVLayout(E, 16, 2, 64, 64)
    pool, table, lens = lay.pool(3, gpu), _i([[0], [1]], gpu), _i([1, 1], gpu)
    f = lambda *s, dtype=BF: torch.randn(*s, device=gpu).to(dtype)  # noqa: E731
    q = f(2, 4, 64)
    for bad in (dict(q=f(2, 4, 128)), dict(q=f(4, 64)), dict(q=f(2, 4, 64, dtype=torch.float16)), dict(q=f(2, 4, 128)[..., ::2]), dict(lens=lens[:1]),
                dict(lens=lens.long()), dict(o=f(2, 4, 32)), dict(o=f(2, 1, 4, 64)), dict(rows=_i([0], gpu)), dict(workspace=f(8)), dict(pool=pool[:, :16]),
                dict(layout=lay._replace(page_tokens=32)), dict(q=q.cpu()), dict(o_dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_attn_decode(**{**dict(q=q, pool=pool, layout=lay, table=table, lens=lens), **bad})
    for bad, word in ((dict(q=f(2, 3, 64)), "SHAPE"), (dict(q=f(2, 17, 4, 64)), "SHAPE"), (dict(o=q), "ALIAS"), (dict(scale=math.inf), "SHAPE"),
                      (dict(q=f(3, 4, 64), lens=_i([1, 1, 1], gpu)), "SHAPE")):
        with pytest.raises(kda.KdaError, match=word):
            kda.kda_attn_decode(**{**dict(q=q, pool=pool, layout=lay, table=table, lens=lens), **bad})
