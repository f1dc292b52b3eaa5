"""kda_qk_norm against the formula in 64 bits: types, norms, head sizes, strided rows, rotations, far positions,
values that are not finite, in place, and a replayed graph."""
import numpy as np
import pytest
import torch

import serving_model as sm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _host(x):
    return None if x is None else x.detach().double().cpu().numpy()


def _check(x, y, out, what, **kw):
    ref, slack = sm.head_norm(_host(x), **kw)
    sm.within(_host(y), ref, slack, sm.HALF_STEP[out], what)


def _freq(rot, gpu):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().to(gpu)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("d,rot,pairing", [(8, 0, "halves"), (16, 16, "halves"), (24, 16, "pairs"), (64, 32, "halves"), (96, 96, "pairs"),
                                           (128, 64, "halves"), (128, 128, "pairs"), (192, 64, "halves"), (256, 256, "halves")])
def test_against_the_formula(gpu, dtype, out, norm, d, rot, pairing):
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(d + rot)
    n, hq, hk = 37, 5, 2
    q = torch.randn(n, hq, d, generator=g, device=gpu).to(DT[dtype])
    k = torch.randn(n, hk, d, generator=g, device=gpu).to(DT[dtype])
    qw, kw = torch.randn(d, generator=g, device=gpu), torch.randn(d, generator=g, device=gpu)
    pos = torch.randint(-5, 1 << 20, (n,), generator=g, device=gpu, dtype=torch.int32)
    fr = _freq(rot, gpu) if rot else None
    yq, yk = kda.kda_qk_norm(q, k, norm=norm, q_weight=qw, k_weight=kw, eps=1e-5, q_scale=0.125, positions=pos if rot else None,
                             inv_freq=fr, pairing=pairing, out_dtype=DT[out])
    assert yq.dtype == DT[out] and yq.shape == q.shape and yk.shape == k.shape
    a = dict(norm=norm, eps=1e-5, positions=_host(pos), inv_freq=_host(fr), pairing=pairing)
    _check(q, yq, out, "q", weight=_host(qw), scale=0.125, **a)
    _check(k, yk, out, "k", weight=_host(kw), **a)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 1023, 1024, 1025, 16385])
@pytest.mark.parametrize("hq,hk,d", [(1, 0, 16), (3, 1, 64), (32, 32, 128)])
def test_lengths(gpu, n, hq, hk, d):
    if n > 2000 and hq > 3:
        n = 2049  # (the oracle's time)
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(n)
    q = torch.randn(n, hq, d, generator=g, device=gpu).to(torch.bfloat16)
    k = torch.randn(n, hk, d, generator=g, device=gpu).to(torch.bfloat16) if hk else None
    pos, fr = torch.arange(n, device=gpu, dtype=torch.int32), _freq(16, gpu)
    yq, yk = kda.kda_qk_norm(q, k, positions=pos, inv_freq=fr)
    a = dict(norm="l2", eps=1e-6, positions=_host(pos), inv_freq=_host(fr))
    _check(q, yq, "bf16", "q", **a)
    if hk:
        _check(k, yk, "bf16", "k", **a)
    else:
        assert yk is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_fused_rows_in_place(gpu, dtype):
    """Queries and keys inside the rows of a fused projection, normalised where they stand: the values beside
    them (and the projection's other columns) keep their bits."""
    kda = _kda()
    n, hq, hk, d = 33, 4, 2, 64
    g = torch.Generator(device=gpu).manual_seed(3)
    rows = torch.randn(n, hq + 2 * hk + 1, d, generator=g, device=gpu).to(DT[dtype])
    before = rows.clone()
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    q0, k0 = q.clone(), k.clone()
    yq, yk = kda.kda_qk_norm(q, k, q_out=q, k_out=k, norm="rms", eps=1e-6)
    assert yq.data_ptr() == rows.data_ptr()
    _check(q0, q, dtype, "q", norm="rms", eps=1e-6)
    _check(k0, k, dtype, "k", norm="rms", eps=1e-6)
    assert torch.equal(rows[:, hq + hk:], before[:, hq + hk:])
    # [B,T,H,d] and [n,H,d] are the same rows; fresh outputs are dense
    r4 = before.reshape(3, 11, -1, d)
    y4, _ = kda.kda_qk_norm(r4[:, :, :hq], r4[:, :, hq:hq + hk], norm="rms", eps=1e-6)
    assert y4.shape == (3, 11, hq, d) and y4.is_contiguous() and torch.equal(y4.reshape(n, hq, d), q)


def test_far_positions(gpu):
    """Angles of positions to 2^31 - 1 and below zero keep their precision."""
    kda = _kda()
    pos = torch.tensor([0, 1, -1, 4096, 10 ** 6, -10 ** 6, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=gpu)
    g = torch.Generator(device=gpu).manual_seed(9)
    q = torch.randn(len(pos), 2, 128, generator=g, device=gpu)
    fr = _freq(128, gpu)
    for pairing in ("halves", "pairs"):
        y, _ = kda.kda_qk_norm(q, positions=pos, inv_freq=fr, pairing=pairing)
        _check(q, y, "f32", pairing, norm="l2", eps=1e-6, positions=_host(pos), inv_freq=_host(fr), pairing=pairing)


def test_values_that_are_not_finite_stay_in_their_head(gpu):
    kda = _kda()
    q = torch.ones(4, 3, 32, device=gpu)
    q[0, 1, 5] = float("nan")
    q[1, 2, 0] = float("inf")
    q[2, 0] = 0.0
    q[3, 0] = 1e-30  # its squares are below fp32's range
    y, _ = kda.kda_qk_norm(q, eps=1e-6)
    want = torch.full_like(q, 1.0 / np.sqrt(32 + 1e-6))
    ok = torch.ones(4, 3, dtype=torch.bool, device=gpu)
    ok[0, 1] = ok[1, 2] = ok[2, 0] = ok[3, 0] = False
    assert torch.allclose(y[ok], want[ok], rtol=1e-6, atol=0)
    assert torch.isnan(y[0, 1]).all()
    assert torch.isnan(y[1, 2, 0]) and (y[1, 2, 1:] == 0).all()
    assert (y[2, 0] == 0).all()
    assert torch.allclose(y[3, 0], torch.full((32,), 1e-27, device=gpu), rtol=1e-5, atol=0)
    z, _ = kda.kda_qk_norm(q[2:3, 0:1], eps=0.0)
    assert torch.isnan(z).all()


def test_no_tokens_and_one_token_of_any_stride(gpu):
    kda = _kda()
    q = torch.empty(0, 4, 64, device=gpu)
    y, _ = kda.kda_qk_norm(q)
    assert y.shape == (0, 4, 64)
    row = torch.randn(1, 9, 64, device=gpu)
    y, _ = kda.kda_qk_norm(row[:, 2:5])
    _check(row[:, 2:5], y, "f32", "one token", norm="l2", eps=1e-6)


def test_graph_replays(gpu):
    kda = _kda()
    n, h, d = 64, 4, 128
    q = torch.randn(n, h, d, device=gpu).to(torch.bfloat16)
    pos, fr = torch.arange(n, device=gpu, dtype=torch.int32), _freq(64, gpu)
    out = torch.empty_like(q)
    kda.kda_qk_norm(q, positions=pos, inv_freq=fr, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_qk_norm(q, positions=pos, inv_freq=fr, q_out=out)
    for i in range(3):
        q.copy_(torch.randn(n, h, d, device=gpu))
        pos.add_(100)
        graph.replay()
        want, _ = kda.kda_qk_norm(q, positions=pos, inv_freq=fr)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
