"""CPU checks of the attention layers' boundary: every refusal returns the documented status before any HIP call (the
pointers are fake, aligned addresses that are never touched), the binding refuses what does not fit, and the plain models
keep their own rules."""
import ctypes
import math

import pytest
import torch

import attention_model as am

BASE = 1 << 40


def _lib():
    import gated_delta_rule_07_amd as kda
    if not kda.library_path().exists():
        pytest.skip("libkda.so not built")
    return kda.load_library()


def _a(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 36) + off)


FWD = dict(q=_a(0), qs=4096, k=_a(1), ks=1024, v=_a(2), vs=1024, dt=1, scale=0.1, cu=_a(3), cuk=_a(4), N=3, nq=100, nk=120, o=_a(5), os=4096,
           odt=1, hq=32, hk=8, dk=128, dv=128)


def _fwd(lib, **over):
    return lib.kda_attn_fwd(*{**FWD, **over}.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), 3), (dict(odt=2), 3), (dict(dt=-1), 3),
    (dict(N=0), 2), (dict(nq=-1), 2), (dict(nk=-1), 2), (dict(nq=(1 << 22) + 1), 2), (dict(hq=0), 2), (dict(hk=0), 2), (dict(hq=12), 2),
    (dict(hq=8192, hk=1), 2), (dict(scale=math.nan), 2), (dict(scale=math.inf), 2), (dict(qs=4088), 2), (dict(ks=1016), 2),
    (dict(os=0), 2), (dict(vs=1 << 62), 2),
    (dict(cu=None, cuk=None, nq=100), 2), (dict(cuk=None), 2), (dict(nq=1 << 22, nk=1 << 22, hq=128, hk=128, qs=1 << 16), 2),
    (dict(dk=96), 4), (dict(dv=256), 4), (dict(dk=0), 4),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(cu=None), 1),
    (dict(q=_a(0, 8)), 5), (dict(cu=_a(3, 4)), 5), (dict(ks=1028), 5), (dict(odt=0, os=4098), 5),
    (dict(o=_a(0)), 6), (dict(o=_a(1, 1024)), 6), (dict(o=_a(2)), 6), (dict(o=_a(3)), 6), (dict(o=_a(4)), 6),
    (dict(nq=0), 0), (dict(nq=0, q=None, k=None, v=None, o=None), 0),
])
def test_fwd_refusals(over, code):
    assert _fwd(_lib(), **over) == code


APP = dict(k=_a(0), ks=1024, v=_a(1), vs=1024, q=_a(2), qs=4096, dt=1, pos=_a(3), fr=_a(4), rot=64, pair=0, qo=_a(5), qos=4096, ko=_a(6),
           kos=1024, pool=_a(7), kv=2, P=64, pt=64, table=_a(8), R=9, W=20, rows=_a(9), lens=_a(10), cu=_a(11), N=5, n=100, hq=32, hk=8, dk=128,
           dv=128)


def _app(lib, **over):
    return lib.kda_kv_append(*{**APP, **over}.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), 3), (dict(kv=0), 3), (dict(kv=3), 3), (dict(pair=2), 3),
    (dict(n=-1), 2), (dict(n=(1 << 22) + 1), 2), (dict(cu=None), 2), (dict(N=0), 2), (dict(N=4097), 2), (dict(P=0), 2), (dict(P=65537), 2),
    (dict(R=0), 2), (dict(W=0), 2), (dict(R=1 << 14, W=1 << 13), 2), (dict(R=1, W=1 << 26, pt=128), 2), (dict(rows=None, N=10), 2), (dict(hk=0), 2),
    (dict(hq=12), 2), (dict(ks=1016), 2), (dict(qos=4088), 2), (dict(vs=-1024), 2),
    (dict(pt=48), 4), (dict(pt=256), 4), (dict(dk=32), 4), (dict(dv=16), 4), (dict(rot=24), 4), (dict(rot=144), 4), (dict(rot=-16), 4),
    (dict(k=None), 1), (dict(v=None), 1), (dict(qo=None), 1), (dict(q=None), 1), (dict(fr=None), 1), (dict(pool=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1),
    (dict(pool=_a(7, 8)), 5), (dict(rows=_a(9, 4)), 5), (dict(lens=_a(10, 4)), 5), (dict(ks=1028), 5), (dict(pos=_a(3, 4)), 5),
    (dict(pool=_a(0)), 6), (dict(pool=_a(8, -16)), 6), (dict(pool=_a(9)), 6), (dict(pool=_a(10)), 6), (dict(pool=_a(11)), 6), (dict(qo=_a(0)), 6),
    (dict(qo=_a(2), qos=8192), 6), (dict(ko=_a(0), kos=2048), 6), (dict(ko=_a(1)), 6), (dict(ko=_a(5)), 6), (dict(ko=_a(7, 128)), 6),
    (dict(ko=_a(3)), 6), (dict(qo=_a(8)), 6),
    (dict(n=0), 0), (dict(n=0, k=None, v=None), 0),
])
def test_append_refusals(over, code):
    assert _app(_lib(), **over) == code


READ = dict(pool=_a(0), kv=1, P=64, pt=64, table=_a(1), R=9, W=20, rows=_a(2), st=_a(3), cu=_a(4), ko=_a(5), vo=_a(6), odt=1, N=5, n=100, hk=8,
            dk=128, dv=64)


@pytest.mark.parametrize("over,code", [
    (dict(odt=2), 3), (dict(kv=0), 3), (dict(n=-1), 2), (dict(N=0), 2), (dict(P=0), 2), (dict(rows=None, N=10), 2), (dict(hk=5000), 2),
    (dict(pt=8), 4), (dict(dk=16), 4), (dict(pool=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(ko=None), 1), (dict(vo=None), 1),
    (dict(st=_a(3, 4)), 5), (dict(ko=_a(5, 8)), 5), (dict(ko=_a(0)), 6), (dict(vo=_a(5, 16)), 6), (dict(vo=_a(1)), 6), (dict(ko=_a(3)), 6),
    (dict(n=0), 0),
])
def test_read_refusals(over, code):
    assert _lib().kda_kv_read(*{**READ, **over}.values(), None) == code


DEC = dict(q=_a(0), dt=1, scale=0.1, pool=_a(1), kv=2, P=64, pt=64, table=_a(2), R=9, W=200, rows=_a(3), lens=_a(4), o=_a(5), odt=1, ws=_a(6),
           wn=1 << 30, B=5, K=2, hq=32, hk=8, dk=128, dv=128)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), 3), (dict(odt=2), 3), (dict(kv=0), 3), (dict(B=0), 2), (dict(B=4097), 2), (dict(K=0), 2), (dict(K=17), 2), (dict(hq=31), 2),
    (dict(scale=math.inf), 2), (dict(wn=1000), 2), (dict(R=1, W=1 << 25, pt=64), 2), (dict(R=5, rows=None, B=6), 2),
    (dict(R=1, W=1 << 20, pt=128, B=4096), 2), (dict(B=4096, K=16, hq=512), 2), (dict(B=1025, hq=4096, K=1, R=2000), 2),
    (dict(pt=24), 4), (dict(dv=32), 4), (dict(q=None), 1), (dict(lens=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(pool=None), 1),
    (dict(q=_a(0, 8)), 5), (dict(ws=_a(6, 8)), 5), (dict(o=_a(0)), 6), (dict(o=_a(1)), 6), (dict(ws=_a(5)), 6), (dict(ws=_a(1)), 6), (dict(o=_a(4)), 6),
    (dict(ws=_a(2)), 6),
])
def test_decode_refusals(over, code):
    assert _lib().kda_attn_decode(*{**DEC, **over}.values(), None) == code


def test_plan_and_page_bytes():
    import gated_delta_rule_07_amd as kda
    _lib()
    for dt, e in ((torch.bfloat16, 2), (torch.float8_e4m3fn, 1)):
        for pt in (16, 32, 64, 128):
            lay = kda.KVLayout(dt, pt, 3, 128, 64)
            assert lay.page_bytes == 3 * pt * 192 * e + (32 if e == 1 else 0) and lay.page_bytes % 16 == 0
            k, v, s = lay.views(lay.pool(5, "cpu"))
            assert k.shape == (5, 3, pt, 128) and v.shape == (5, 3, pt, 64) and (s is None) == (e == 2)
            assert kda.kda_attn_decode_plan(lay, 4, 1, 6, 1) == 0 and kda.kda_attn_decode_plan(lay, 4, 1, 6, 1 << 14) > 0
    for bad in (kda.KVLayout(torch.float16, 64, 3, 128, 64), kda.KVLayout(torch.bfloat16, 64, 0, 128, 64),
                kda.KVLayout(torch.bfloat16, 65, 3, 128, 64), kda.KVLayout(torch.bfloat16, 64, 3, 96, 64)):
        with pytest.raises(kda.KdaError):
            bad.page_bytes
    lib = _lib()
    n = ctypes.c_size_t(0)
    assert lib.kda_kv_page_bytes(1, 64, 1, 64, 64, None) == 1
    for args, code in (((0, 64, 9, 1, 1, 8, 8, 64, 64), 3), ((1, 64, 9, 0, 1, 8, 8, 64, 64), 2), ((1, 64, 9, 1, 17, 8, 8, 64, 64), 2),
                       ((1, 64, 1 << 25, 1, 1, 8, 8, 64, 64), 2), ((1, 64, 9, 1, 1, 8, 3, 64, 64), 2), ((1, 64, 9, 1, 1, 8, 8, 32, 64), 4)):
        assert lib.kda_attn_decode_plan(*args, ctypes.byref(n)) == code
    assert lib.kda_attn_decode_plan(1, 64, 9, 1, 1, 8, 8, 64, 64, None) == 1


def test_cpu_tensors_are_refused():
    import gated_delta_rule_07_amd as kda
    _lib()
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    lay = kda.KVLayout(torch.bfloat16, 16, 2, 64, 64)
    one = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: kda.kda_attn_fwd(x, x, x), lambda: kda.kda_kv_append(x, x, lay.pool(2, "cpu"), lay, one[None], one),
                 lambda: kda.kda_kv_read(lay.pool(2, "cpu"), lay, one[None], one, 3), lambda: kda.kda_attn_decode(x, lay.pool(2, "cpu"), lay, one[None], one)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


# ---- the models' own rules ------------------------------------------------------------------------


def test_e4m3_model_is_the_format():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    fine = codes[torch.isfinite(codes)]
    assert torch.equal(am.e4m3(fine), fine) and float(fine.max()) == 448.0
    x = torch.linspace(-448, 448, 100003, dtype=torch.float64)
    x = torch.cat([x, x / 2.0 ** 12, x / 2.0 ** 16]).float().double()  # (PyTorch rounds to e4m3 by way of fp32)
    assert torch.equal(am.e4m3(x), x.to(torch.float8_e4m3fn).double())
    s = torch.sort(fine).values
    mid = (s[1:] + s[:-1]) / 2
    assert torch.equal(am.e4m3(mid), mid.float().to(torch.float8_e4m3fn).double())
    assert torch.isnan(am.e4m3(torch.tensor([math.inf, -math.inf, math.nan], dtype=torch.float64))).all()


@pytest.mark.parametrize("amax,e", [(0.0, -100), (448.0, 0), (448.0001, 1), (1.75, -8), (1.7500001, -7), (1.0, -8), (3e38, 120), (1e-40, -100)])
def test_scale_model(amax, e):
    assert am.scale_of(amax) == 2.0 ** e


def test_attention_model():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, 2, 16, generator=g, dtype=torch.float64) for n in (7, 9, 9))
    o, slack = am.fwd(q, k, v, 0.3, [7], [9])
    mask = torch.full((7, 9), -math.inf, dtype=torch.float64).triu(3)
    for h in range(2):
        want = torch.softmax(q[:, h] @ k[:, h].T * 0.3 + mask, -1) @ v[:, h]
        assert float((o[:, h] - want).abs().max()) < 1e-14
    assert 0 < float(slack.max()) < 1e-3
    v[5:] = math.nan  # what a query does not see does not reach it
    o2, _ = am.fwd(q, k, v, 0.3, [7], [9])
    assert float((o2[:3] - o[:3]).abs().max()) < 1e-14 and torch.isnan(o2[3:]).all()  # (sums of 5 products in another order)
    o3, _ = am.fwd(q, k[:2], v[:2], 0.3, [7], [2])
    assert not o3[:5].any() and o3[5:].any()
    with pytest.raises(AssertionError):
        am.close((o + 3 * slack).float(), o, slack * 0.0)


def test_turn_model():
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    f = torch.tensor([0.5, 0.25] * 4)
    for pairing in ("halves", "pairs"):
        y, _ = am.turn(x, [0, 7, -2], f, pairing)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 16:], x[..., 16:])
        back, _ = am.turn(y, [0, -7, 2], f, pairing)
        assert float((back - x).abs().max()) < 1e-14
    a, b = x[1, 0, 0], x[1, 0, 8]
    y, _ = am.turn(x, [0, 7, -2], f, "halves")
    assert abs(float(y[1, 0, 0] - (a * math.cos(3.5) - b * math.sin(3.5)))) < 1e-14
