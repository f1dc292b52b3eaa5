"""CPU checks of the serving calls' boundary: every refusal returns the documented status before any HIP call (the
pointers are fake, aligned addresses that are never touched), the Python binding refuses what it should, and the
plain models that the GPU tests compare with keep their own rules."""
import ctypes
import random

import numpy as np
import pytest
import torch

import serving_model as sm

BASE = 1 << 40


def _lib():
    import gated_delta_rule_07_amd as kda
    if not kda.library_path().exists():
        pytest.skip("libkda.so not built")
    return kda.load_library()


def _a(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 36) + off)


def _norm(lib, **over):
    a = dict(q=_a(0), qs=1024, k=_a(1), ks=512, dt=1, norm=0, qw=_a(2), kw=_a(3), eps=1e-6, scale=1.0, pos=_a(4), fr=_a(5),
             rot=64, pair=0, qo=_a(6), qos=1024, ko=_a(7), kos=512, odt=1, n=100, hq=8, hk=4, d=128)
    a.update(over)
    return lib.kda_qk_norm(*[a[x] for x in ("q", "qs", "k", "ks", "dt", "norm", "qw", "kw", "eps", "scale", "pos", "fr", "rot", "pair",
                                            "qo", "qos", "ko", "kos", "odt", "n", "hq", "hk", "d")], None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), 3), (dict(odt=-1), 3), (dict(norm=2), 3), (dict(pair=7), 3),
    (dict(n=-1), 2), (dict(hq=0), 2), (dict(hk=-1), 2), (dict(n=2 ** 31 - 1, hq=2 ** 20), 2),
    (dict(eps=-1e-6), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2),
    (dict(qs=1016), 2), (dict(kos=0), 2), (dict(ks=-512), 2), (dict(qs=1 << 62), 2),
    (dict(d=12), 4), (dict(d=264), 4), (dict(d=0), 4), (dict(rot=24), 4), (dict(rot=144), 4), (dict(rot=-16), 4),
    (dict(q=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(fr=None), 1),
    (dict(q=_a(0, 8)), 5), (dict(qw=_a(2, 4)), 5), (dict(qs=1028), 5), (dict(odt=0, kos=514), 5),
    (dict(qo=_a(0), qos=2048), 6), (dict(qo=_a(0), odt=0), 6), (dict(qo=_a(1)), 6), (dict(ko=_a(6, 256)), 6),
    (dict(ko=_a(4)), 6), (dict(qo=_a(0, 16)), 6),
    # outputs between the rows of one wider array: side by side is fine, one value too many is not
    (dict(q=_a(0), qs=4096, qo=_a(0, 2 * 1016), qos=4096), 6), (dict(q=_a(0), qs=4096, qo=_a(0, 2 * 3080), qos=4096), 6),
    (dict(q=_a(0), qs=4096, qo=_a(0, 2 * 1024), qos=2048), 6),
    (dict(n=0), 0), (dict(n=0, q=None), 0),
])
def test_norm_refusals(over, code):
    assert _norm(_lib(), **over) == code


def _fork(lib, **over):
    a = dict(table=_a(0), ref=_a(1), par=_a(2), ch=_a(3), moves=_a(4), nm=_a(5), n=8, priv=1, R=32, W=4, P=64)
    a.update(over)
    return lib.kda_cache_fork(*[a[x] for x in ("table", "ref", "par", "ch", "moves", "nm", "n", "priv", "R", "W", "P")], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 2), (dict(n=1025), 2), (dict(priv=-1), 2), (dict(priv=5), 2), (dict(R=0), 2), (dict(W=0), 2), (dict(P=0), 2),
    (dict(P=65537), 2), (dict(R=1 << 20, W=65), 2),
    (dict(table=None), 1), (dict(ref=None), 1), (dict(par=None), 1), (dict(ch=None), 1), (dict(moves=None), 1), (dict(nm=None), 1),
    (dict(par=_a(2, 4)), 5), (dict(nm=_a(5, 8)), 5),
    (dict(par=_a(0)), 6), (dict(moves=_a(1, 240)), 6), (dict(nm=_a(4, 48)), 6), (dict(ref=_a(0, 496)), 6), (dict(ch=_a(4, 16)), 6),
])
def test_fork_refusals(over, code):
    assert _fork(_lib(), **over) == code


@pytest.mark.parametrize("args,code", [
    ((_a(0), _a(1), _a(2), -1, 8, 2, 9), 2), ((_a(0), _a(1), _a(2), 1, 8, 0, 9), 2), ((_a(0), _a(1), _a(2), 1 << 30, 8, 8, 9), 2),
    ((None, _a(1), _a(2), 1, 8, 2, 9), 1), ((_a(0), _a(1), None, 1, 8, 2, 9), 1), ((_a(0), _a(1), _a(2, 4), 1, 8, 2, 9), 5),
    ((_a(0), _a(0, 48), _a(2), 1, 8, 2, 9), 6), ((_a(0), _a(1), _a(1, 32), 1, 8, 2, 9), 6), ((_a(0), _a(1), None, 0, 8, 2, 9), 0),
])
def test_free_refusals(args, code):
    assert _lib().kda_cache_free(*args, None) == code


def _compact(lib, **over):
    a = dict(t=_a(0), r=_a(1), to=_a(2), ro=_a(3), m=_a(4), nm=_a(5), nl=_a(6), R=32, W=4, P=64)
    a.update(over)
    return lib.kda_cache_compact(*[a[x] for x in ("t", "r", "to", "ro", "m", "nm", "nl", "R", "W", "P")], None)


@pytest.mark.parametrize("over,code", [
    (dict(R=0), 2), (dict(P=65537), 2), (dict(W=-1), 2), (dict(to=None), 1), (dict(nl=None), 1), (dict(m=_a(4, 8)), 5),
    (dict(to=_a(0, 16)), 6), (dict(ro=_a(0)), 6), (dict(m=_a(1, 128)), 6), (dict(nl=_a(4, 240)), 6), (dict(to=_a(1)), 6),
])
def test_compact_refusals(over, code):
    assert _compact(_lib(), **over) == code


def _copy(lib, **over):
    a = dict(src=_a(0), dst=_a(0), page=4096, L=2, ns=16, nd=16, m=_a(1), nm=_a(2), most=8)
    a.update(over)
    return lib.kda_cache_copy(*[a[x] for x in ("src", "dst", "page", "L", "ns", "nd", "m", "nm", "most")], None)


@pytest.mark.parametrize("over,code", [
    (dict(page=0), 2), (dict(L=0), 2), (dict(ns=0), 2), (dict(nd=65537), 2), (dict(most=-1), 2), (dict(most=65537), 2),
    (dict(page=1 << 36, L=65536, nd=65536, ns=65536), 2), (dict(src=None), 1), (dict(m=None), 1),
    (dict(page=4104), 5), (dict(dst=_a(0, 8)), 5),
    (dict(dst=_a(0, 4096)), 6), (dict(ns=8), 6), (dict(m=_a(0, 4096)), 6), (dict(nm=_a(0, 16)), 6), (dict(most=0), 0),
])
def test_copy_refusals(over, code):
    assert _copy(_lib(), **over) == code


def _decode(lib, **over):
    a = dict(q=_a(0), k=_a(1), v=_a(2), dt=1, alpha=_a(3), z=None, A=None, beta=_a(4), pool=_a(5), P=9, pi=_a(6), po=_a(7), o=_a(8),
             odt=0, B=4, H=2, dk=128, dv=128)
    a.update(over)
    return lib.kda_decode_step_paged(*[a[x] for x in ("q", "k", "v", "dt", "alpha", "z", "A", "beta", "pool", "P", "pi", "po", "o",
                                                      "odt", "B", "H", "dk", "dv")], None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), 3), (dict(odt=9), 3), (dict(B=0), 2), (dict(B=4097), 2), (dict(H=0), 2), (dict(P=0), 2), (dict(P=65537), 2),
    (dict(B=4096, H=1025), 2), (dict(dk=48), 4), (dict(dv=256), 4), (dict(alpha=None), 1), (dict(alpha=None, z=_a(3)), 1), (dict(pi=None), 1), (dict(o=None), 1),
    (dict(pool=None), 1), (dict(pi=_a(6, 4)), 5), (dict(o=_a(5, 1 << 16)), 6), (dict(o=_a(6)), 6), (dict(po=_a(5)), 6),
    (dict(q=_a(5, 16)), 6), (dict(alpha=None, z=_a(3), A=_a(8)), 6),
])
def test_decode_refusals(over, code):
    assert _decode(_lib(), **over) == code


def _verify(lib, **over):
    a = dict(q=_a(0), k=_a(1), v=_a(2), dt=1, alpha=_a(3), beta=_a(4), pool=_a(5), P=9, pages=_a(6), par=_a(7), nn=_a(8), o=_a(9),
             odt=0, u=_a(10), B=4, K=16, H=2, dk=128, dv=128)
    a.update(over)
    return lib.kda_tree_verify(*[a[x] for x in ("q", "k", "v", "dt", "alpha", "beta", "pool", "P", "pages", "par", "nn", "o", "odt",
                                                "u", "B", "K", "H", "dk", "dv")], None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=5), 3), (dict(odt=2), 3), (dict(B=0), 2), (dict(K=0), 2), (dict(K=65), 2), (dict(H=-1), 2), (dict(P=0), 2),
    (dict(pages=None, P=3), 2), (dict(B=1 << 12, H=1025), 2),
    (dict(K=64, H=1 << 17), 2), (dict(dk=24), 4), (dict(dv=8), 4), (dict(par=None), 1), (dict(u=None), 1), (dict(alpha=None), 1),
    (dict(u=_a(10, 4)), 5), (dict(u=_a(9)), 6), (dict(o=_a(5)), 6), (dict(u=_a(3)), 6), (dict(o=_a(7, 128)), 6),
])
def test_verify_refusals(over, code):
    assert _verify(_lib(), **over) == code


def _commit(lib, **over):
    a = dict(k=_a(1), dt=1, alpha=_a(3), u=_a(10), par=_a(7), nn=_a(8), last=_a(9), pool=_a(5), P=9, pi=_a(6), po=_a(11), B=4, K=16,
             H=2, dk=128, dv=128)
    a.update(over)
    return lib.kda_tree_commit(*[a[x] for x in ("k", "dt", "alpha", "u", "par", "nn", "last", "pool", "P", "pi", "po", "B", "K", "H",
                                                "dk", "dv")], None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=3), 3), (dict(B=4097), 2), (dict(K=65), 2), (dict(P=0), 2), (dict(pi=None, P=3), 2), (dict(B=4096, H=1025), 2), (dict(dk=100), 4),
    (dict(last=None), 1), (dict(u=None), 1), (dict(last=_a(9, 8)), 5), (dict(u=_a(5)), 6), (dict(last=_a(5, 64)), 6),
    (dict(po=_a(5, 1024)), 6),
])
def test_commit_refusals(over, code):
    assert _commit(_lib(), **over) == code


def test_binding_refusals():
    import gated_delta_rule_07_amd as kda
    q = torch.zeros(2, 3, 16)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_qk_norm(q)
    with pytest.raises(TypeError):
        kda.kda_qk_norm(None)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_cache_fork(i.view(2, 2), i, i, i)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_cache_free(i.view(2, 2), i, i)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_cache_compact(i.view(2, 2), i)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_cache_copy(q, i.view(2, 2))
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_decode_step_paged(q, q, q, q, q, q, i)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_tree_verify(q, q, q, q, q, q, i, i)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kda_tree_commit(q, q, q, i, i, q, i)


def test_argument_helper_agrees_with_its_python_form():
    """The compiled check refuses what the Python form refuses, with its words."""
    import gated_delta_rule_07_amd as kda
    helper = pytest.importorskip("gated_delta_rule_07_amd._kda_args")
    assert kda._need is helper.need
    seen = []
    helper.set_refuse(lambda *a: seen.append(a) or 7)
    try:
        x = torch.zeros(2, 3)
        cases = [(x, "x", torch.float32, 0, (2, 3)), (None, "x", torch.float32, 0, (2, 3)), (x, "x", "f32", 0, (2, 3)),
                 (x.to_sparse(), "x", torch.float32, 0, (2, 3)), (torch.empty(2, 3, device="meta"), "x", torch.float32, 0, (2, 3)),
                 (x, "x", torch.float32, 0, (2, "3")), (x, "x", torch.float32, 0, [2, 3])]
        for a in cases:
            assert helper.need(*a) == 7 and seen[-1] == a
        with pytest.raises(TypeError):
            helper.need(x, "x")
    finally:
        helper.set_refuse(kda._need_in_words)
    with pytest.raises(ValueError, match="HIP device"):
        kda._need(x, "x", torch.float32, 0, (2, 3))


# ---- the models -----------------------------------------------------------------------------------


@pytest.mark.parametrize("seed", range(20))
def test_model_of_the_cache_keeps_its_books(seed):
    """Through random forks, frees and packings the refs stay the number of entries that hold each page, and the
    pages' contents follow the rows."""
    rng = random.Random(seed)
    P, R, W = rng.randint(4, 40), rng.randint(2, 12), rng.randint(1, 4)
    table, ref = [[-1] * W for _ in range(R)], [0] * P
    pool, held = np.zeros((1, P, 1)), {}
    for turn in range(30):
        if rng.random() < 0.5:
            n = rng.randint(1, 4)
            par, ch = [rng.randint(-1, R - 1) for _ in range(n)], [rng.randrange(R) for _ in range(n)]
            before = [list(r) for r in table]
            table, ref, moves = sm.fork(table, ref, par, ch, rng.randint(0, W))
            pool = sm.copy(pool, pool, moves, True)
            for p, c in zip(par, ch):
                if table[c] != before[c] and c not in held:
                    held[c] = held[p] if p >= 0 else [0.0] * W
            for r in range(R):  # decode: a page that one entry holds gets a new state
                if ref[table[r][0]] == 1 and table[r][0] >= 0:
                    pool[0, table[r][0]] = turn + r / 100
                    held[r] = [turn + r / 100] + held[r][1:]
        elif rng.random() < 0.6:
            rows = [rng.randrange(R) for _ in range(2)]
            table, ref = sm.free(table, ref, rows)
            for r in rows:
                held.pop(r, None)
        else:
            table, ref, moves, live = sm.compact(table, ref)
            pool = sm.copy(pool, pool, moves, True)
            assert all(r <= 0 for r in ref[live:])
        for page in range(P):
            assert ref[page] == sum(r.count(page) for r in table)
        for r in held:
            for w in range(W):
                if table[r][w] >= 0:
                    assert pool[0, table[r][w], 0] == held[r][w]


def test_model_of_a_tree_equals_the_oracle():
    """A chain run by the tree's model is the oracle's recurrence."""
    import kda_inputs as ki
    import oracle
    x = ki.make_prefill(1, 12, 1, 16, 32, torch.float32, 3.0, 0.1, seed=4)
    ro, rs = oracle.forward(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S0"])
    h = {n: t.double().numpy() for n, t in x.items()}
    r = sm.tree_run(h["S0"][0, 0], h["q"][0, :, 0], h["k"][0, :, 0], h["v"][0, :, 0], h["alpha"][0, :, 0], h["beta"][0, :, 0],
                    list(range(-1, 11)))
    assert np.abs(r["o"] - ro[0]).max() < 1e-12 and np.abs(r["states"][-1] - rs[0]).max() < 1e-12
    assert r["depth"] == list(range(1, 13))


def test_models_reject_nan():
    with pytest.raises(AssertionError):
        sm.within([float("nan")], [1.0], np.ones(1), 1.0)
