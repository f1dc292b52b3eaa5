"""kda_kv_append and kda_kv_read against plain models in 64 bits: types, page sizes, positions, groups, padding, pages that
are out of range or shared, scales that grow, values that are not finite, far pages, graphs."""
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


def _cu(lens, gpu):
    return _i([sum(lens[:i]) for i in range(len(lens) + 1)], gpu)


def _filled(kda, lay, P, gpu, seed):
    """A pool of codes and scales that are all finite numbers."""
    g = torch.Generator(device=gpu).manual_seed(seed)
    pool = lay.pool(P, gpu)
    k, v, s = lay.views(pool)
    for x in (k, v):
        x.copy_(torch.randn(x.shape, generator=g, device=gpu).mul_(20 if lay.dtype == E else 1).to(x.dtype))
    if s is not None:
        s.copy_(torch.exp2(torch.randint(-9, 0, s.shape, generator=g, device=gpu).float()))
    return pool


def _tables(lay, need, gpu, seed, extra=4):
    """(table, page lists) of rows that hold need[b] pages each, in random order."""
    g = torch.Generator().manual_seed(seed)
    P = sum(need) + extra
    order = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b + 1])], dtype=torch.int32)
    return P, table.to(gpu)


def _same_pages(lay, pool, want, slack=None):
    """The pool holds what the model's pages do: bit for bit, or (slack: of each [keys, values] of a page) as roundings of
    values within slack."""
    got = am.Pages(lay, pool)
    for i in range(2):
        if got.scales is not None:
            assert torch.equal(got.scales[:, i], want.scales[:, i]), "scales"
        x, y = got.kv[i], want.kv[i]
        assert torch.equal(torch.isnan(x), torch.isnan(y)), "NaN"
        x, y = torch.nan_to_num(x), torch.nan_to_num(y)
        if slack is None:
            assert torch.equal(x, y), f"{int((x != y).sum())} values differ"
            continue
        # a value within slack of y rounds to y's code or the next one, and to the next one only where y is that near to the border
        if got.scales is None:
            tol = 2.0 ** -7 * y.abs() + 1e-37
        else:
            tol = torch.maximum(2.0 ** -3 * y.abs(), torch.tensor(2.0 ** -9))
        assert bool(((x - y).abs() <= tol).all())
        assert float((x != y).double().mean()) <= slack, "too many values at another code"


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("pt", [16, 32, 64, 128])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_without_rotation_bit_for_bit(gpu, dtype, cache, pt, dk, dv):
    """Lengths that begin and end anywhere, empty ones, a bf16 or fp32 input: pages equal the model's exactly."""
    kda = _kda()
    lay = kda.KVLayout(cache, pt, 3, dk, dv)
    before, lens = [0, 5, pt, 2 * pt - 1, 40, 0, 7, 3 * pt], [1, 130, pt, 2, 0, 3 * pt + 5, 1, 17]
    P, table = _tables(lay, [-(-(a + n) // pt) for a, n in zip(before, lens)], gpu, 1)
    pool = _filled(kda, lay, P, gpu, 2)
    g = torch.Generator(device=gpu).manual_seed(3)
    n = sum(lens)
    k, v = (torch.randn(n, 3, d, generator=g, device=gpu).mul(3).to(dtype) for d in (dk, dv))
    k[:, 1] *= 2.0 ** -30  # (a head whose scale stays what the page's earlier tokens need)
    want = am.Pages(lay, pool)
    split = lambda x: list(x.cpu().to(BF).double().split(lens)) if cache == BF else list(x.cpu().double().split(lens))  # noqa: E731
    want.append(table.tolist(), before, split(k), split(v))
    kda.kda_kv_append(k, v, pool, lay, table, _i(before, gpu), cu_seqlens=_cu(lens, gpu))
    torch.cuda.synchronize()
    _same_pages(lay, pool, want)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("pairing", ["halves", "pairs"])
@pytest.mark.parametrize("dk,rot", [(64, 16), (64, 64), (128, 128), (128, 48)])
def test_rotation(gpu, dtype, cache, pairing, dk, rot):
    kda = _kda()
    lay = kda.KVLayout(cache, 32, 2, dk, 64)
    before, lens = [900001, 3, 0, 33], [70, 1, 40, 31]
    need = [-(-(a + n) // 32) for a, n in zip(before, lens)]
    before[0], need[0] = 900001 % 32, 4  # (its positions are given: far into a context)
    P, table = _tables(lay, need, gpu, 4)
    pool = _filled(kda, lay, P, gpu, 5)
    g = torch.Generator(device=gpu).manual_seed(6)
    n = sum(lens)
    q, k, v = (torch.randn(n, h, d, generator=g, device=gpu).to(dtype) for h, d in ((6, dk), (2, dk), (2, 64)))
    freq = 10000.0 ** (-torch.arange(rot // 2, device=gpu).float() / (rot // 2))
    pos = [a + i for a, m in zip([900001, 3, 0, 33], lens) for i in range(m)]
    want = am.Pages(lay, pool)
    tk, sk = am.turn(k.cpu(), pos, freq, pairing)
    tq, sq = am.turn(q.cpu(), pos, freq, pairing)
    rounded = tk.to(BF).double() if cache == BF else tk
    want.append(table.tolist(), before, list(rounded.split(lens)), list((v.cpu().to(BF) if cache == BF else v.cpu()).double().split(lens)))
    ko = torch.zeros_like(k)
    qo, ko2 = kda.kda_kv_append(k, v, pool, lay, table, _i(before, gpu), cu_seqlens=_cu(lens, gpu), q=q, inv_freq=freq,
                                positions=_i(pos, gpu), pairing=pairing, k_out=ko)
    torch.cuda.synchronize()
    assert ko2 is ko
    am.close(qo, tq, sq, "q_out")
    am.close(ko, tk, sk, "k_out")
    # fp32 may put a value at the next code where the 64-bit one lies within 32 u (|a| + |b|) of the border between two codes: for values near 1 and
    # steps of 2^-8 and more that is one in 2^8 / (2 * 32 * 2^-24 * 4) = 2^17; ten times that for the small values
    _same_pages(lay, pool, want, slack=1e-3)


@pytest.mark.parametrize("cache", [BF, E])
def test_one_token_each(gpu, cache):
    """A decode batch with padding and places of their own; the same token again changes nothing."""
    kda = _kda()
    lay = kda.KVLayout(cache, 16, 4, 64, 64)
    N, before = 9, [0, 1, 15, 16, 17, 31, 32, 100, 5]
    P, table = _tables(lay, [b // 16 + 1 for b in before], gpu, 7)
    pool = _filled(kda, lay, P, gpu, 8)
    rows = [8, 7, -1, 5, 4, 3, 99, 1, 0]
    g = torch.Generator(device=gpu).manual_seed(9)
    k, v = (torch.randn(N, 4, 64, generator=g, device=gpu).to(BF) for _ in range(2))
    want = am.Pages(lay, pool)
    t = table.tolist()
    lens = [before[r] if 0 <= r < 9 else 3 for r in rows]
    want.append([t[r] if 0 <= r < 9 else None for r in rows], lens, list(k.cpu().double().split(1)), list(v.cpu().double().split(1)))
    for _ in range(2):
        kda.kda_kv_append(k, v, pool, lay, table, _i(lens, gpu), rows=_i(rows, gpu))
        torch.cuda.synchronize()
        _same_pages(lay, pool, want)


def test_a_page_that_fills_token_by_token(gpu):
    """A page of growing, shrinking, zero, tiny, huge and not finite tokens, one call each: scales only grow."""
    kda = _kda()
    lay = kda.KVLayout(E, 16, 2, 64, 64)
    pool = _filled(kda, lay, 2, gpu, 10)
    table = _i([[1]], gpu)
    g = torch.Generator(device=gpu).manual_seed(11)
    want = am.Pages(lay, pool)
    sizes = [0.0, 1e-30, 1.0, 3.0, 0.1, 448.0, 448.01, 1e-38, 7e4, 0.0, math.nan, math.inf, 3e38, 1.0, 1e30, -5.0]
    for t, size in enumerate(sizes):
        k, v = (torch.randn(1, 2, 64, generator=g, device=gpu).clamp(-1, 1) * size for _ in range(2))
        k[0, 0, 3], v[0, 1, 5] = size, size
        kda.kda_kv_append(k, v, pool, lay, table, _i([t], gpu))
        want.append([[1]], [t], [k.cpu().double()], [v.cpu().double()])
        torch.cuda.synchronize()
        _same_pages(lay, pool, want)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("table,before,lens,rows", [
    ([[0, 1], [1, 2]], [16, 0], [3, 2], None),               # a page of two sequences: neither writes it
    ([[0, 1, 0], [2, 3, 4]], [0, 5], [40, 20], None),        # a page twice in a row
    ([[0], [1], [2]], [3, 3, 3], [1, 1, 1], [1, 1, 2]),      # one row twice
    ([[-1, 9], [99, 2 ** 31 - 1]], [3, 0], [20, 20], None),  # out of range
    ([[0, 1], [2, 3]], [30, -9], [5, 4], None),              # behind the row's end; a negative length
    ([[3, 0], [1, 2]], [2 ** 31 - 1, 31], [5, 4], None),
    ([[i] for i in range(5)] + [[4]] * 70, [2] * 75, [1] * 75, None),  # more sequences than a wave has lanes
    ([[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 0], [10] * 11], [0, 0], [170, 3], None),  # many pages of one sequence
])
def test_pages_that_may_not_be_written(gpu, cache, table, before, lens, rows):
    kda = _kda()
    lay = kda.KVLayout(cache, 16, 2, 64, 64)
    pool = _filled(kda, lay, 11, gpu, 12)
    g = torch.Generator(device=gpu).manual_seed(13)
    n = sum(lens)
    k, v = (torch.randn(n, 2, 64, generator=g, device=gpu).to(BF) for _ in range(2))
    want = am.Pages(lay, pool)
    want.append([table[r] for r in (rows or range(len(lens)))], [max(b, 0) for b in before], list(k.cpu().double().split(lens)), list(v.cpu().double().split(lens)))
    ko, freq = torch.full_like(k, 7.0), torch.zeros(8, device=gpu)
    kda.kda_kv_append(k, v, pool, lay, _i(table, gpu), _i(before, gpu), rows=None if rows is None else _i(rows, gpu), cu_seqlens=_cu(lens, gpu),
                      inv_freq=freq, k_out=ko)
    torch.cuda.synchronize()
    _same_pages(lay, pool, want)
    assert torch.equal(ko, k)  # (a rotation by nothing; tokens that are not stored have their rows too)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("lens,same", [
    ([700], [(0, 3, 0, 40)]),                                                      # a page early and late in one row
    ([350, 20, 400], [(0, 18, 2, 24), (2, 1, 1, 0)]),                              # among pages behind the sixteenth, and before it
    ([300, 310, 17, 330, 290, 500, 280], [(1, 17, 5, 30), (4, 2, 6, 16), (0, 16, 0, 17)]),  # more long sequences than waves
    ([40] * 70 + [600, 1, 320], [(70, 37, 3, 1), (72, 19, 69, 2), (71, 0, 70, 5)]),        # sequences behind the 64th
])
def test_shared_pages_of_long_sequences(gpu, cache, lens, same):
    kda = _kda()
    lay = kda.KVLayout(cache, 16, 2, 64, 64)
    need = [-(-(n + 5) // 16) for n in lens]
    P, table = _tables(lay, need, gpu, 32)
    for b, i, c, j in same:
        table[c, j] = table[b, i]
    pool = _filled(kda, lay, P, gpu, 33)
    g = torch.Generator(device=gpu).manual_seed(34)
    k, v = (torch.randn(sum(lens), 2, 64, generator=g, device=gpu).to(BF) for _ in range(2))
    want = am.Pages(lay, pool)
    want.append(table.tolist(), [5] * len(lens), list(k.cpu().double().split(lens)), list(v.cpu().double().split(lens)))
    kda.kda_kv_append(k, v, pool, lay, table, _i([5] * len(lens), gpu), cu_seqlens=_cu(lens, gpu))
    _same_pages(lay, pool, want)


def test_lists_that_are_wrong(gpu):
    """Offsets that decrease or lie out of range: nothing out of range is touched, rows outside every sequence are left."""
    kda = _kda()
    for cache in (BF, E):
        lay = kda.KVLayout(cache, 16, 2, 64, 64)
        pool = _filled(kda, lay, 8, gpu, 14)
        table = _i([[0, 1], [2, 3], [4, 5]], gpu)
        k = torch.ones(40, 2, 64, device=gpu, dtype=BF)
        for cu in ([30, 10, 20, 40], [-5, 2 ** 31 - 1, -2 ** 31, 7], [100, 100, 100, 100]):
            kda.kda_kv_append(k, k, pool, lay, table, _i([2 ** 31 - 1, -2 ** 31, 3], gpu), cu_seqlens=_i(cu, gpu), q=k)
            kda.kda_kv_read(pool, lay, table, _i(cu, gpu), 40, starts=_i([2 ** 31 - 1, -2 ** 31, 30], gpu))
        q, qo = torch.ones(40, 4, 64, device=gpu, dtype=BF), torch.full((40, 4, 64), 7.0, device=gpu, dtype=BF)
        ko = torch.full_like(k, 7.0)
        kda.kda_kv_append(k, k, pool, lay, table, _i([0, 0, 0], gpu), cu_seqlens=_i([5, 9, 9, 30], gpu), q=q, q_out=qo, k_out=ko)
        for x in (qo, ko):
            assert bool((x[:5] == 7).all()) and bool((x[5:30] == 1).all()) and bool((x[30:] == 7).all())
        a, _ = kda.kda_kv_append(k, k, pool, lay, table, _i([0, 0, 0], gpu), cu_seqlens=_i([5, 9, 9, 30], gpu), q=q)
        assert not a[:5].any() and not a[30:].any() and bool((a[5:30] == 1).all())
    torch.cuda.synchronize()


def test_in_place_and_strides(gpu):
    """Rows of a fused projection, queries and keys turned in place."""
    kda = _kda()
    lay = kda.KVLayout(BF, 16, 2, 64, 64)
    g = torch.Generator(device=gpu).manual_seed(15)
    row = torch.randn(21, 8, 64, generator=g, device=gpu).to(BF)
    q, k, v = row[:, :4], row[:, 4:6], row[:, 6:]
    P, table = _tables(lay, [2], gpu, 16)
    freq = torch.tensor([1.0, 0.1] * 8, device=gpu)
    pool, dense = lay.pool(P, gpu), lay.pool(P, gpu)
    qo, _ = kda.kda_kv_append(k.contiguous(), v.contiguous(), dense, lay, table, _i([0], gpu), cu_seqlens=_i([0, 21], gpu), q=q.contiguous(), inv_freq=freq)
    was = row.clone()
    kda.kda_kv_append(k, v, pool, lay, table, _i([0], gpu), cu_seqlens=_i([0, 21], gpu), q=q, inv_freq=freq, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(pool, dense) and torch.equal(row[:, :4], qo) and torch.equal(row[:, 6:], was[:, 6:])
    ko, vo = kda.kda_kv_read(pool, lay, table, _i([0, 21], gpu), 21)
    assert torch.equal(ko, row[:, 4:6]) and torch.equal(vo, row[:, 6:])


def test_a_page_of_128_with_a_full_rotation(gpu):
    """The largest table of cosines and sines."""
    kda = _kda()
    lay = kda.KVLayout(E, 128, 1, 128, 128)
    pool, table = lay.pool(4, gpu), _i([[2, 0, 3]], gpu)
    g = torch.Generator(device=gpu).manual_seed(17)
    k, v = (torch.randn(300, 1, 128, generator=g, device=gpu) for _ in range(2))
    freq = 10000.0 ** (-torch.arange(64, device=gpu).float() / 64)
    want = am.Pages(lay, pool)
    tk, _ = am.turn(k.cpu(), list(range(300)), freq, "halves")
    want.append([[2, 0, 3]], [0], [tk], [v.cpu().double()])
    kda.kda_kv_append(k, v, pool, lay, table, _i([0], gpu), cu_seqlens=_i([0, 300], gpu), inv_freq=freq)
    torch.cuda.synchronize()
    _same_pages(lay, pool, want, slack=1e-3)


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("out", [BF, F])
@pytest.mark.parametrize("pt,dk,dv", [(16, 64, 64), (64, 128, 64), (128, 64, 128)])
def test_read(gpu, cache, out, pt, dk, dv):
    kda = _kda()
    lay = kda.KVLayout(cache, pt, 3, dk, dv)
    lens, starts = [1, 0, 2 * pt + 3, 7, pt, 50], [0, 3, pt - 1, 2 * pt, 5, -4]
    need = [-(-(max(a, 0) + n) // pt) for a, n in zip(starts, lens)]
    P, table = _tables(lay, need, gpu, 18)
    table[2, 1] = -1
    table[5, 0] = P
    pool = _filled(kda, lay, P, gpu, 19)
    rows = [0, 1, 2, -1, 4, 5]
    n = sum(lens) + 4  # (rows behind the last sequence)
    ko, vo = torch.full((n, 3, dk), 7.0, device=gpu, dtype=out), torch.full((n, 3, dv), 7.0, device=gpu, dtype=out)
    kda.kda_kv_read(pool, lay, table, _cu(lens, gpu), n, rows=_i(rows, gpu), starts=_i(starts, gpu), k_out=ko, v_out=vo)
    m, t, at = am.Pages(lay, pool), table.tolist(), 0
    for b, ln in enumerate(lens):
        a = max(starts[b], 0)
        k, v, there = m.tokens(t[rows[b]] if rows[b] >= 0 else [], a + ln)
        for got, ref in ((ko, k), (vo, v)):
            x = torch.where(there[a:, None, None], ref[a:], 7.0)
            assert torch.equal(got[at:at + ln].double().cpu(), x), f"sequence {b}"
        at += ln
    assert bool((ko[at:] == 7).all()) and bool((vo[at:] == 7).all())
    ko, vo = kda.kda_kv_read(pool, lay, table, _cu(lens, gpu), n, rows=_i(rows, gpu), starts=_i(starts, gpu), out_dtype=out)
    assert ko.dtype == vo.dtype == out and not ko[at:].any() and not vo[at:].any()


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("out", [BF, F])
def test_read_of_more_rows_than_a_cache_holds(gpu, cache, out):
    """As many rows as are stored past the caches: those of calls with few rows each."""
    kda = _kda()
    lay = kda.KVLayout(cache, 64, 5, 128, 64)
    lens = [150001, 1, 4444, 77]
    P, table = _tables(lay, [-(-n // 64) for n in lens], gpu, 30)
    table[0, 1000] = -1
    pool = _filled(kda, lay, P, gpu, 31)
    n = sum(lens) + 3
    ko, vo = torch.full((n, 5, 128), 7.0, device=gpu, dtype=out), torch.full((n, 5, 64), 7.0, device=gpu, dtype=out)
    assert (ko.numel() + vo.numel()) * ko.element_size() > 256 << 20
    kda.kda_kv_read(pool, lay, table, _cu(lens, gpu), n, k_out=ko, v_out=vo)
    at = 0
    for b, ln in enumerate(lens):
        for a in range(0, ln, 30000):
            m = min(30000, ln - a)
            x, y = torch.full((m, 5, 128), 7.0, device=gpu, dtype=out), torch.full((m, 5, 64), 7.0, device=gpu, dtype=out)
            kda.kda_kv_read(pool, lay, table, _i([0, m], gpu), m, rows=_i([b], gpu), starts=_i([a], gpu), k_out=x, v_out=y)
            assert torch.equal(ko[at + a:at + a + m], x) and torch.equal(vo[at + a:at + a + m], y), (b, a)
        at += ln
    assert bool((ko[at:] == 7).all()) and bool((vo[at:] == 7).all())


def test_far_pages(gpu):
    """Pages that start past 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    kda = _kda()
    lay = kda.KVLayout(E, 128, 64, 128, 128)
    P = 2100
    pool = torch.empty(P, lay.page_bytes, dtype=torch.uint8, device=gpu)
    assert (P - 3) * lay.page_bytes > 2 ** 32
    g = torch.Generator(device=gpu).manual_seed(20)
    k, v = (torch.randn(140, 64, 128, generator=g, device=gpu).to(BF) for _ in range(2))
    small, table = lay.pool(3, gpu), _i([[P - 1, P - 2]], gpu)
    kda.kda_kv_append(k, v, pool, lay, table, _i([0], gpu), cu_seqlens=_i([0, 140], gpu))
    kda.kda_kv_append(k, v, small, lay, _i([[2, 1]], gpu), _i([0], gpu), cu_seqlens=_i([0, 140], gpu))
    a, b = kda.kda_kv_read(pool, lay, table, _i([0, 140], gpu), 140), kda.kda_kv_read(small, lay, _i([[2, 1]], gpu), _i([0, 140], gpu), 140)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and float((a[0].float() - k.float()).abs().max()) <= 2.0 ** -4 * 8


def test_many_sequences(gpu):
    """As many as a call takes, one of whose pages is shared with the last."""
    kda = _kda()
    lay = kda.KVLayout(E, 16, 1, 64, 64)
    N = 4096
    pool = _filled(kda, lay, N, gpu, 21)
    table = torch.arange(N, device=gpu, dtype=torch.int32)[:, None].contiguous()
    table[17] = N - 1
    g = torch.Generator(device=gpu).manual_seed(22)
    k, v = (torch.randn(N, 1, 64, generator=g, device=gpu).to(BF) for _ in range(2))
    lens = torch.arange(N, device=gpu, dtype=torch.int32) % 16
    old = pool.clone()
    want = am.Pages(lay, pool)
    want.append(table.tolist(), lens.tolist(), list(k.cpu().double().split(1)), list(v.cpu().double().split(1)))
    kda.kda_kv_append(k, v, pool, lay, table, lens)
    torch.cuda.synchronize()
    _same_pages(lay, pool, want)
    assert torch.equal(pool[N - 1], old[N - 1]) and torch.equal(pool[17], old[17])


def test_captured(gpu):
    """An append and a read, replayed on new tokens, lengths and rows."""
    kda = _kda()
    lay = kda.KVLayout(E, 16, 2, 64, 64)
    P, table = _tables(lay, [6, 6, 6], gpu, 23)
    pool = _filled(kda, lay, P, gpu, 24)
    other = pool.clone()
    g = torch.Generator(device=gpu).manual_seed(25)
    k, v, q = (torch.randn(40, h, 64, generator=g, device=gpu).to(BF) for h in (2, 2, 4))
    freq = torch.tensor([1.0, 0.1] * 8, device=gpu)
    lens, cu, rows = _i([0, 0, 0], gpu), _i([0, 10, 20, 40], gpu), _i([0, 1, 2], gpu)
    qo, ko, vo = torch.zeros_like(q), torch.zeros(90, 2, 64, device=gpu, dtype=BF), torch.zeros(90, 2, 64, device=gpu, dtype=BF)
    cu_read = _i([0, 30, 60, 90], gpu)
    bufs = [x.clone() for x in (qo, ko, vo)]

    def step(pool, qo, ko, vo):
        kda.kda_kv_append(k, v, pool, lay, table, lens, rows=rows, cu_seqlens=cu, q=q, inv_freq=freq, q_out=qo)
        kda.kda_kv_read(pool, lay, table, cu_read, 90, rows=rows, k_out=ko, v_out=vo)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(pool, qo, ko, vo)
    for i, (ln, c, r) in enumerate((([0, 0, 0], [0, 10, 20, 40], [0, 1, 2]), ([10, 10, 20], [0, 1, 2, 3], [0, 1, 2]), ([11, 11, 0], [0, 30, 30, 40], [2, -1, 0]))):
        lens.copy_(_i(ln, gpu)), cu.copy_(_i(c, gpu)), rows.copy_(_i(r, gpu)), k.mul_(-1.5)
        graph.replay()
        step(other, *bufs)
        torch.cuda.synchronize()
        assert torch.equal(pool, other) and all(torch.equal(a, b) for a, b in zip((qo, ko, vo), bufs)), f"replay {i}"


def test_binding_refusals(gpu):
    kda = _kda()
    lay = kda.KVLayout(E, 16, 2, 64, 64)
    pool, table, lens = lay.pool(3, gpu), _i([[0], [1]], gpu), _i([0, 0], gpu)
    f = lambda *s, dtype=BF: torch.randn(*s, device=gpu).to(dtype)  # noqa: E731
    k = f(2, 2, 64)
    for bad in (dict(k=f(2, 3, 64)), dict(v=f(2, 2, 128)), dict(v=f(3, 2, 64)), dict(k=f(2, 2, 64, dtype=F)), dict(pool=lay.pool(3, gpu)[:, :-16]),
                dict(pool=pool.float()), dict(layout=lay._replace(dtype=F)), dict(table=table.long()), dict(table=table[0]), dict(lens=lens[:1]),
                dict(rows=_i([0], gpu)), dict(cu_seqlens=_i([0, 1], gpu).float()), dict(q=f(2, 4, 32)), dict(q=f(3, 4, 64)), dict(q_out=k),
                dict(inv_freq=f(8)), dict(inv_freq=f(8, dtype=F), positions=_i([1], gpu)), dict(pairing="both"), dict(k_out=f(2, 2, 32)), dict(k=k.cpu())):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_kv_append(**{**dict(k=k, v=k, pool=pool, layout=lay, table=table, lens=lens), **bad})
    for bad, word in ((dict(v=k, k_out=k), "ALIAS"), (dict(inv_freq=f(4, dtype=F)), "UNSUPPORTED"), (dict(inv_freq=f(40, dtype=F)), "UNSUPPORTED"),
                      (dict(q=f(2, 3, 64)), "SHAPE"), (dict(k=f(0, 2, 64), v=f(0, 2, 64), lens=lens[:0]), "SHAPE")):
        with pytest.raises((kda.KdaError), match=word):
            kda.kda_kv_append(**{**dict(k=k, v=k.clone() if "k_out" not in bad else k, pool=pool, layout=lay, table=table, lens=lens), **bad})
    cu = _i([0, 1, 2], gpu)
    for bad in (dict(cu_seqlens=cu.long()), dict(k_out=f(2, 2, 32)), dict(k_out=k, v_out=f(2, 2, 64, dtype=F)), dict(out_dtype=torch.float16), dict(starts=cu),
                dict(total=3, k_out=k)):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_kv_read(**{**dict(pool=pool, layout=lay, table=table, cu_seqlens=cu, total=2), **bad})
