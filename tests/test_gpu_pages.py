"""The cache of state pages (kda_cache_fork, _free, _compact, _copy) against plain models of their rules: every
table, reference count, move list and page equal."""
import random

import numpy as np
import pytest
import torch

import serving_model as sm

pytestmark = pytest.mark.gpu


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu, shape=None):
    t = torch.tensor(x, dtype=torch.int32)
    return (t if shape is None else t.reshape(shape)).to(gpu)


def _cache(rng, P, R, W, rows_used, shared):
    """A consistent table and refs: some rows use pages of their own in slot 0, and share recorded ones."""
    order = list(range(P))
    rng.shuffle(order)
    table, ref = [[-1] * W for _ in range(R)], [0] * P
    for r in rng.sample(range(R), rows_used):
        if not order:
            break
        table[r][0] = order.pop()
        for w in range(1, W):
            if shared and rng.random() < 0.6:
                table[r][w] = rng.choice(shared)
            elif order and rng.random() < 0.5:
                table[r][w] = order.pop()
        for p in table[r]:
            if p >= 0:
                ref[p] += 1
    return table, ref


def _fork_equal(gpu, table, ref, parents, children, n_private):
    kda = _kda()
    t, f = _i(table, gpu), _i(ref, gpu)
    moves, n = kda.kda_cache_fork(t, f, _i(parents, gpu), _i(children, gpu), n_private)
    wt, wf, wm = sm.fork(table, ref, parents, children, n_private)
    assert t.tolist() == wt
    assert f.tolist() == wf
    assert int(n) == len(wm) and [tuple(m) for m in moves[:len(wm)].tolist()] == wm
    return wt, wf, wm


@pytest.mark.parametrize("seed", range(12))
def test_fork(gpu, seed):
    rng = random.Random(seed)
    P, R, W = rng.choice([1, 5, 64, 1023, 1025, 3000]), rng.choice([2, 9, 70]), rng.randint(1, 5)
    table, ref = _cache(rng, P, R, W, R // 2, list(range(0, P, 7)))
    n = rng.choice([1, 3, R, 2 * R])
    _fork_equal(gpu, table, ref, [rng.randint(-1, R - 1) for _ in range(n)], [rng.randint(0, R - 1) for _ in range(n)],
                rng.randint(0, W))


def test_fork_refusals(gpu):
    """Lists out of range, a child in use, a child named twice (by a fork that could not start it too), a child as
    its own parent and as another's, a table with pages out of range."""
    table = [[3, 9, -7], [-1, -1, 99], [0, 100, 5], [-1] * 3, [-1] * 3, [-1] * 3, [100, -1, -1]]
    ref = [1, 0, 0, 1, 0, 1, 0, 0, 0, 1]
    parents = [0, 7, 0, -2, 0, 2, 2, 3, 4, 0, 1, -1, 0]
    children = [2, 3, 7, 3, 3, 4, 4, 5, 5, -1, 1, 6, 6]
    _fork_equal(gpu, table, ref, parents, children, 2)
    _fork_equal(gpu, table, ref, [], [], 2)
    _fork_equal(gpu, table, ref, [0, 0], [3, 4], 0)


def test_fork_until_the_pages_run_out(gpu):
    table = [[0, 1], [2, -1]] + [[-1, -1] for _ in range(6)]
    ref = [1, 1, 1, 0, -3, 0]
    _fork_equal(gpu, table, ref, [0, 1, -1, 1, 1], [2, 3, 4, 5, 6], 2)
    _fork_equal(gpu, table, [1] * 6, [0, 1], [2, 3], 1)
    _fork_equal(gpu, table, [1] * 6, [0, 1], [2, 3], 0)


def test_fork_most(gpu):
    """1024 forks at once over a pool of 65536 pages."""
    R, P = 2048, 65536
    ref = [1 if p % 3 or p < 700 else 0 for p in range(P)]
    table = [[r, r + 1] for r in range(1024)] + [[-1, -1] for _ in range(1024)]
    _fork_equal(gpu, table, ref, [(7 * i) % 1024 for i in range(1024)], [1024 + (5 * i) % 1024 for i in range(1024)], 1)


@pytest.mark.parametrize("seed", range(6))
def test_free(gpu, seed):
    kda = _kda()
    rng = random.Random(seed)
    P, R, W = rng.choice([1, 40, 500]), rng.choice([1, 30, 300]), rng.randint(1, 9)
    table, ref = _cache(rng, P, R, W, R, list(range(0, P, 5)))
    if seed % 2:
        table[0][0], ref[P // 2] = P + 3, 0  # a page that does not exist; a count that is too low
    rows = [rng.randint(-2, R + 1) for _ in range(rng.randint(1, 2 * R))]
    t, f = _i(table, gpu), _i(ref, gpu)
    kda.kda_cache_free(t, f, _i(rows, gpu))
    wt, wf = sm.free(table, ref, rows)
    assert t.tolist() == wt and f.tolist() == wf


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,R,W,frac", [(1, 1, 1, 1.0), (2, 3, 2, 0.5), (97, 48, 2, 0.3), (1024, 40, 3, 0.0), (1025, 9, 1, 1.0),
                                        (5000, 700, 5, 0.6), (65536, 30000, 1, 0.5)])
def test_compact(gpu, in_place, P, R, W, frac):
    kda = _kda()
    rng = random.Random(P)
    ref = [rng.randint(1, 3) if rng.random() < frac else -rng.randint(0, 1) for _ in range(P)]
    table = [[rng.randint(-2, P) for _ in range(W)] for _ in range(R)]  # (some free, some out of range)
    t, f = _i(table, gpu), _i(ref, gpu)
    to, fo, moves, n, live = kda.kda_cache_compact(t, f, table_out=t if in_place else None, ref_out=f if in_place else None)
    wt, wf, wm, wl = sm.compact(table, ref)
    assert int(live) == wl and int(n) == len(wm)
    assert [tuple(m) for m in moves[:len(wm)].tolist()] == wm
    assert to.tolist() == wt and fo.tolist() == wf
    if not in_place:
        assert t.tolist() == table and f.tolist() == ref


def _copy_equal(gpu, layers, P, shape, moves, n_moves=None, src_pages=None, dtype=torch.float32):
    kda = _kda()
    lead = () if layers is None else (layers,)
    make = lambda pages: (100 * torch.randn(*lead, pages, *shape)).to(dtype)  # noqa: E731
    pool, src = make(P), None if src_pages is None else make(src_pages)
    d, s = pool.to(gpu), None if src is None else src.to(gpu)
    m = _i(moves, gpu, (len(moves), 2))
    kda.kda_cache_copy(d, m, None if n_moves is None else _i([n_moves], gpu), src=s, n_layers=layers)
    n = len(moves) if n_moves is None else min(max(n_moves, 0), len(moves))
    view = lambda x: (x if layers is not None else x[None]).float().numpy()  # noqa: E731
    want = sm.copy(view(pool if src is None else src), view(pool), moves[:n], src is None)
    assert np.array_equal(view(d.cpu()), want)
    if s is not None:
        assert torch.equal(s.cpu(), src)


@pytest.mark.parametrize("layers,shape", [(None, (2, 16, 16)), (3, (1, 4)), (2, (3, 64, 64)), (1, (32, 128, 128)), (5, (1, 1028))])
def test_copy(gpu, layers, shape):
    """Pages of 16 bytes to 2 MiB, whole tiles and not; a page forked to several; zeros; moves past the count."""
    moves = [(0, 5), (0, 6), (1, 7), (-1, 8), (2, 2), (9, 3)]
    _copy_equal(gpu, layers, 11, shape, moves)
    _copy_equal(gpu, layers, 11, shape, moves, n_moves=2)
    _copy_equal(gpu, layers, 11, shape, moves, n_moves=0)
    _copy_equal(gpu, layers, 11, shape, moves, n_moves=-4)
    _copy_equal(gpu, layers, 11, shape, moves, n_moves=99)


def test_copy_passes_over_moves_that_race(gpu):
    """Two moves onto one page, a chain, a swap, pages out of range: none of them runs, the others do."""
    moves = [(0, 4), (1, 4), (2, 5), (5, 6), (7, 8), (8, 7), (3, 9), (10, 11), (11, 10), (-2, 1), (0, 12), (12, 0), (3, -1), (9, 9)]
    _copy_equal(gpu, None, 12, (2, 32, 32), moves)
    _copy_equal(gpu, 2, 12, (2, 32, 32), [(3, 1), (3, 1), (4, 2)])
    _copy_equal(gpu, None, 12, (2, 32, 32), [(5, 5), (5, 6)])


def test_copy_between_pools(gpu):
    """From a smaller and a larger pool; a page of the same number is no move onto itself there."""
    moves = [(0, 0), (1, 5), (5, 1), (3, 2), (-1, 4)]
    _copy_equal(gpu, 2, 6, (2, 16, 64), moves, src_pages=9)
    _copy_equal(gpu, None, 9, (2, 16, 64), moves, src_pages=4, dtype=torch.bfloat16)


def test_copy_many_small_pages(gpu):
    rng = random.Random(1)
    P = 65536
    pages = rng.sample(range(P), 60000)
    _copy_equal(gpu, None, P, (4,), list(zip(pages[:30000], pages[30000:])) + [(pages[0], pages[30000])])


def test_fork_and_copy_replayed(gpu):
    """A fork, its copies and the free captured in one graph: each replay reads the lists as they are then."""
    kda = _kda()
    P, R, W = 40, 12, 2
    table = [[r, 30 + r] for r in range(4)] + [[-1, -1] for _ in range(R - 4)]
    ref = [1 if p < 4 or 30 <= p < 34 else 0 for p in range(P)]
    pool = torch.randn(2, P, 3, 16, 16)
    t, f, d = _i(table, gpu), _i(ref, gpu), pool.to(gpu)
    parents, children, ends = _i([0, 0, 1], gpu), _i([4, 5, 6], gpu), _i([0], gpu)
    moves, n = _i([[0, 0]] * 3, gpu), _i([0], gpu)

    def step():
        kda.kda_cache_fork(t, f, parents, children, 1, moves=moves, n_moves=n)
        kda.kda_cache_copy(d, moves, n, n_layers=2)
        kda.kda_cache_free(t, f, ends)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    host = pool.numpy()
    for par, chi, end in (([0, 0, 1], [4, 5, 6], [0]), ([4, 5, 2], [0, 7, 8], [5]), ([7, -1, 8], [5, 9, 10], [4])):
        parents.copy_(_i(par, gpu)), children.copy_(_i(chi, gpu)), ends.copy_(_i(end, gpu))
        graph.replay()
        torch.cuda.synchronize()
        table, ref, m = sm.fork(table, ref, par, chi, 1)
        host = sm.copy(host, host, m, True)
        table, ref = sm.free(table, ref, end)
        assert t.tolist() == table and f.tolist() == ref and np.array_equal(d.cpu().numpy(), host)
