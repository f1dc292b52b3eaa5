"""kda_attn_fwd against the definition in 64 bits: head sizes, types, groups, strides, packed sequences, prefixes, values
that are not finite where nobody looks, streams and graphs."""
import math

import pytest
import torch

import attention_model as am

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _cu(lens, gpu):
    return _i([sum(lens[:i]) for i in range(len(lens) + 1)], gpu)


def _qkv(gpu, seed, n, m, hq, hk, dk, dv, dtype):
    g = torch.Generator(device=gpu).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=gpu).to(dtype)  # noqa: E731
    return r(n, hq, dk), r(m, hk, dk), r(m, hk, dv)


def _check(q, k, v, lens, lens_k=None, o_dtype=None, scale=None):
    kda, gpu = _kda(), q.device
    o = torch.full((*q.shape[:2], v.shape[2]), 7.0, device=gpu, dtype=o_dtype or q.dtype)
    kda.kda_attn_fwd(q, k, v, scale=scale, cu_seqlens=_cu(lens, gpu), cu_seqlens_k=None if lens_k is None else _cu(lens_k, gpu), o=o)
    ref, slack = am.fwd(q, k, v, q.shape[2] ** -0.5 if scale is None else scale, lens, lens_k)
    am.close(o, ref, slack, "o")
    return o


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_head_sizes(gpu, dtype, dk, dv):
    q, k, v = _qkv(gpu, dk + dv, 149, 149, 4, 2, dk, dv, dtype)
    _check(q, k, v, [149], o_dtype=F)


# Heads: few, so that the waves of a workgroup share the keys, and so many that even one row a sequence makes more workgroups
# than the card holds at once, so that they share the queries.
HEADS = [(4, 2), (258, 2)]


@pytest.mark.parametrize("hq,hk", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513])
def test_lengths(gpu, d, n, hq, hk):
    q, k, v = _qkv(gpu, n, n, n, hq, hk, d, d, BF)
    _check(q, k, v, [n])


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
def test_head_sizes_of_many_heads(gpu, dk, dv):
    q, k, v = _qkv(gpu, dk, 200, 200, 258, 2, dk, dv, BF)
    _check(q, k, v, [200], o_dtype=F)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (6, 2), (10, 2), (16, 1), (40, 8)])
def test_groups(gpu, dtype, hq, hk):
    q, k, v = _qkv(gpu, hq, 130, 130, hq, hk, 64, 64, dtype)
    _check(q, k, v, [130])


@pytest.mark.parametrize("dtype,d,hq", [(BF, 64, 4), (BF, 128, 4), (F, 64, 4), (BF, 32, 4), (BF, 64, 12), (BF, 128, 12)])
def test_packed(gpu, dtype, d, hq):
    lens = [1, 0, 300, 64, 0, 0, 7, 129, 256, 31, 1, 513, 0]
    q, k, v = _qkv(gpu, 3, sum(lens), sum(lens), hq, 2, d, d, dtype)
    _check(q, k, v, lens)


@pytest.mark.parametrize("dtype,d,hq", [(BF, 64, 4), (BF, 128, 4), (F, 128, 4), (BF, 64, 24), (BF, 128, 24)])
def test_prefixes(gpu, dtype, d, hq):
    """More keys than queries, as many, fewer (queries that see nothing give zeros), none."""
    lens, lens_k = [5, 130, 64, 9, 40, 17, 3, 0, 70], [300, 130, 65, 4, 0, 1000, 3, 50, 69]
    q, k, v = _qkv(gpu, 4, sum(lens), sum(lens_k), hq, 2, d, d, dtype)
    o = _check(q, k, v, lens, lens_k)
    a = sum(lens[:3])
    assert not o[a:a + 5].any() and o[a + 5:a + 9].any() and not o[a + 9:a + 49].any()


# Long sequences, and enough heads: on the fp32 matrix cores a workgroup takes 32 queries.
@pytest.mark.parametrize("dtype,dk,dv", [(F, 128, 128), (F, 64, 128), (F, 128, 64), (F, 16, 16), (F, 32, 64), (F, 64, 32), (BF, 32, 16), (BF, 16, 128), (BF, 128, 32)])
@pytest.mark.parametrize("lens,lens_k", [([601, 530, 705], None), ([1, 1500], None), ([40, 301, 5, 200], [900, 300, 700, 650]), ([544], [513])])
def test_long_sequences(gpu, dtype, dk, dv, lens, lens_k):
    q, k, v = _qkv(gpu, 16, sum(lens), sum(lens_k or lens), 16, 4, dk, dv, dtype)
    _check(q, k, v, lens, lens_k)


@pytest.mark.parametrize("dtype,d", [(F, 64), (F, 128), (BF, 32)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_long_sequences_with_values_that_are_not_finite(gpu, dtype, d, bad):
    kda = _kda()
    lens = [600, 530, 700]
    q, k, v = _qkv(gpu, 17, 1830, 1830, 16, 2, d, d, dtype)
    clean = kda.kda_attn_fwd(q, k, v, cu_seqlens=_cu(lens, gpu))
    for t, begin, end in ((0, 0, 600), (599, 0, 600), (600, 600, 1130), (615, 600, 1130), (616, 600, 1130), (631, 600, 1130), (1000, 600, 1130), (1829, 1130, 1830)):
        for x in (k, v):
            y = x.clone()
            y[t, 1, 3] = bad
            o = kda.kda_attn_fwd(q, y if x is k else k, y if x is v else v, cu_seqlens=_cu(lens, gpu))
            same = torch.ones(1830, dtype=torch.bool, device=gpu)
            same[t:end] = False
            assert torch.equal(o[:, :8], clean[:, :8]), "another head"
            # (a tile without the values that are not finite: the same sums)
            assert torch.equal(o[same], clean[same]), f"before token {t}"
            if x is v:
                assert not torch.isfinite(o[t:end, 8:, 3]).any()
                o[t:end, 8:, 3] = clean[t:end, 8:, 3]
                assert torch.equal(o, clean), "another channel"


@pytest.mark.parametrize("dtype,hq", [(BF, 2), (F, 2), (BF, 140)])
def test_long_keys(gpu, dtype, hq):
    q, k, v = _qkv(gpu, 5, 40, 5003, hq, 1, 128, 128, dtype)
    _check(q, k, v, [40], [5003])


# Which kernel runs depends on heads and lengths: queries shared by waves, and keys.
@pytest.mark.parametrize("hq,hk", [(700, 1), (24, 3)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("n,m", [(40, 2003), (257, 1000)])
def test_long_keys_of_many_heads(gpu, hq, hk, dk, dv, n, m):
    q, k, v = _qkv(gpu, 18, n, m, hq, hk, dk, dv, BF)
    _check(q, k, v, [n], [m])


@pytest.mark.parametrize("d,hq,hk", [(128, 8, 1), (128, 16, 4), (64, 8, 8), (64, 16, 2), (128, 40, 8)])
def test_long_prompts(gpu, d, hq, hk):
    q, k, v = _qkv(gpu, 19, 1300, 1300, hq, hk, d, d, BF)
    _check(q, k, v, [1300])
    _check(q, k, v, [1, 1000, 299])


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 32), (F, 64)])
@pytest.mark.parametrize("hq,hk", [(3, 3), (20, 5), (24, 6), (7, 7), (12, 12), (80, 80), (66, 3)])
def test_heads_that_dies_share(gpu, dtype, d, hq, hk):
    """Key heads that do not divide among eight: every tile of every head is somebody's."""
    q, k, v = _qkv(gpu, 20, 711, 711, hq, hk, d, d, dtype)
    _check(q, k, v, [3, 0, 500, 208])


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F, 64)])
def test_strides(gpu, dtype, d):
    """Slices of a fused projection's rows, an output between other rows, [B,T] forms."""
    kda = _kda()
    g = torch.Generator(device=gpu).manual_seed(6)
    rows = torch.randn(2 * 77, 8, d, generator=g, device=gpu).to(dtype)
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    wide = torch.full((2 * 77, 7, d), 3.0, device=gpu, dtype=dtype)
    kda.kda_attn_fwd(q, k, v, cu_seqlens=_cu([77, 77], gpu), o=wide[:, 2:6])
    ref, slack = am.fwd(q, k, v, d ** -0.5, [77, 77])
    am.close(wide[:, 2:6], ref, slack)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 6:] == 3).all())
    o = kda.kda_attn_fwd(*(x.unflatten(0, (2, 77)) for x in (q, k, v)))
    assert o.shape == (2, 77, 4, d) and torch.equal(o.flatten(0, 1), wide[:, 2:6])
    o = kda.kda_attn_fwd(q[:77], k, v)  # one sequence, twice as many keys
    am.close(o, *am.fwd(q[:77], k, v, d ** -0.5, [77], [154]))


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 20.0])
@pytest.mark.parametrize("dtype,hq", [(BF, 2), (F, 2), (BF, 80)])
def test_scales(gpu, dtype, hq, scale):
    q, k, v = _qkv(gpu, 7, 100, 100, hq, 2, 64, 64, dtype)
    if scale == 20.0:  # (scores of hundreds: a softmax that picks one key)
        q, k = (x * 0.5 for x in (q, k))
    _check(q, k, v, [100], scale=scale)


def test_rows_outside_sequences_are_left(gpu):
    kda = _kda()
    for dtype in (BF, F):
        q, k, v = _qkv(gpu, 8, 100, 100, 2, 1, 64, 64, dtype)
        for cu in ([10, 40, 90], [0, 100, 400], [-5, 30, 30]):
            o = torch.full((100, 2, 64), 7.0, device=gpu, dtype=dtype)
            kda.kda_attn_fwd(q, k, v, cu_seqlens=_i(cu, gpu), o=o)
            c = [min(max(x, 0), 100) for x in cu]
            ref, slack = am.fwd(q[c[0]:c[-1]], k[c[0]:c[-1]], v[c[0]:c[-1]], 0.125, [b - a for a, b in zip(c, c[1:])])
            am.close(o[c[0]:c[-1]], ref, slack)
            assert bool((o[:c[0]] == 7).all()) and bool((o[c[-1]:] == 7).all())
        o = kda.kda_attn_fwd(q, k, v, cu_seqlens=_i([10, 40], gpu))
        assert not o[:10].any() and not o[40:].any()
        for cu in ([50, 20, 100], [100, 0, 50], [0, -7, 3], [2 ** 31 - 1, -2 ** 31, 5]):  # wrong lists: nothing out of range
            kda.kda_attn_fwd(q, k, v, cu_seqlens=_i(cu, gpu), cu_seqlens_k=_i([60, 10, 2 ** 30], gpu))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,d,hq", [(BF, 64, 4), (BF, 128, 4), (F, 64, 4), (F, 128, 4), (BF, 32, 4), (BF, 64, 24), (BF, 128, 24)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_query_does_not_see_has_no_influence(gpu, dtype, d, hq, bad):
    kda = _kda()
    lens, G = [100, 70, 300], hq // 2
    q, k, v = _qkv(gpu, 9, 470, 470, hq, 2, d, d, dtype)
    cu = _cu(lens, gpu)
    clean, want = kda.kda_attn_fwd(q, k, v, cu_seqlens=cu), am.fwd(q, k, v, d ** -0.5, lens)
    for t in (99, 100, 135, 169, 170, 200, 469):
        for x in (k, v):
            y = x.clone()
            y[t, 1] = bad
            o = kda.kda_attn_fwd(q, y if x is k else k, y if x is v else v, cu_seqlens=cu)
            b = 0 if t < 100 else 1 if t < 170 else 2
            end = sum(lens[:b + 1])
            same = torch.ones(470, dtype=torch.bool, device=gpu)
            same[t:end] = False
            assert torch.equal(o[:, :G], clean[:, :G]), "another head"
            # (the rows of the tile that holds it may be summed in another order)
            am.close(o[same], *(z[same] for z in want), f"before token {t}")
            if x is v or bad != -math.inf:
                assert not torch.isfinite(o[t:end, G:]).all(-1).all() if x is k else not torch.isfinite(o[t:end, G:]).any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_nothing_to_attend_with_or_to(gpu, dtype):
    kda = _kda()
    q, k, v = _qkv(gpu, 15, 3, 3, 4, 2, 64, 64, dtype)
    assert kda.kda_attn_fwd(q[:0], k, v).shape == (0, 4, 64)
    o = torch.full((3, 4, 64), 7.0, device=gpu, dtype=dtype)
    kda.kda_attn_fwd(q, k[:0], v[:0], o=o)
    assert not o.any()
    kda.kda_attn_fwd(q, k[:0], v[:0], cu_seqlens=_i([0, 2, 3], gpu), cu_seqlens_k=_i([0, 0, 0], gpu), o=o.fill_(7))
    assert not o.any()
    assert kda.kda_attn_fwd(q[:0].unflatten(0, (2, 0)), k[:2].unflatten(0, (2, 1)), v[:2].unflatten(0, (2, 1))).shape == (2, 0, 4, 64)


def test_nothing_but_minus_infinity(gpu):
    """A row all of whose scores are minus infinity gives zeros, as one that sees nothing."""
    kda = _kda()
    for dtype, hq in ((BF, 1), (F, 1), (BF, 300)):
        q, k, v = torch.ones(3, hq, 64, device=gpu, dtype=dtype), torch.full((3, 1, 64), -math.inf, device=gpu, dtype=dtype), torch.ones(3, 1, 64, device=gpu, dtype=dtype)
        assert not kda.kda_attn_fwd(q, k, v).any()
        k[2] = 1.0
        assert kda.kda_attn_fwd(q, k, v)[:, -1, 0].tolist() == [0.0, 0.0, 1.0]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F, 64)])
def test_many_sequences(gpu, dtype, d):
    lens = [(i * 7) % 5 for i in range(3000)]
    n = sum(lens)
    q, k, v = _qkv(gpu, 10, n, n, 2, 1, d, d, dtype)
    kda = _kda()
    o = kda.kda_attn_fwd(q, k, v, cu_seqlens=_cu(lens, gpu))
    some = 700
    am.close(o[:sum(lens[:some])], *am.fwd(q[:sum(lens[:some])], k[:sum(lens[:some])], v[:sum(lens[:some])], d ** -0.5, lens[:some]))
    last = sum(lens[-300:])
    am.close(o[-last:], *am.fwd(q[-last:], k[-last:], v[-last:], d ** -0.5, lens[-300:]))


def test_far_rows(gpu):
    """Rows past 2^32 bytes of q, k and v (slices of wide rows)."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    kda = _kda()
    n, d = 40000, 128
    wide = torch.empty(n, 512, d, device=gpu, dtype=BF)  # 5.2 GB
    assert wide.numel() * 2 > 2 ** 32
    g = torch.Generator(device=gpu).manual_seed(11)
    wide[-200:, :4] = torch.randn(200, 4, d, generator=g, device=gpu).to(BF)
    q, k, v = wide[:, :2], wide[:, 2:3], wide[:, 3:4]
    o = kda.kda_attn_fwd(q, k, v, cu_seqlens=_i([n - 200, n], gpu), o=wide[:, 4:6])
    am.close(o[-200:], *am.fwd(q[-200:], k[-200:], v[-200:], d ** -0.5, [200]))


@pytest.mark.parametrize("dtype,n,hq", [(BF, 2000, 8), (BF, 900, 8), (F, 900, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_repeats_are_bit_equal(gpu, dtype, n, hq, d):
    kda = _kda()
    q, k, v = _qkv(gpu, 12, n, n, hq, 2, d, d, dtype)
    a = kda.kda_attn_fwd(q, k, v)
    for _ in range(5):
        assert torch.equal(kda.kda_attn_fwd(q, k, v), a)


@pytest.mark.parametrize("dtype,hq", [(BF, 4), (BF, 40), (F, 4)])
def test_side_stream_and_graph(gpu, dtype, hq):
    kda = _kda()
    lens = [70, 130, 3]
    q, k, v = _qkv(gpu, 13, 203, 203, hq, 2, 128, 128, dtype)
    cu = _cu(lens, gpu)
    want = kda.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    late = torch.empty_like(q).copy_(q)
    side.wait_stream(torch.cuda.current_stream())
    o = kda.kda_attn_fwd(late, k, v, cu_seqlens=cu, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    graph, o = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        kda.kda_attn_fwd(q, k, v, cu_seqlens=cu, o=o)
    for lens in ([70, 130, 3], [1, 1, 201], [203, 0, 0], [100, 100, 0]):
        cu.copy_(_cu(lens, gpu))
        q.mul_(-1)
        o.fill_(7)
        graph.replay()
        want = torch.full_like(o, 7.0)
        kda.kda_attn_fwd(q, k, v, cu_seqlens=cu, o=want)
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_binding_refusals(gpu):
    kda = _kda()
    q, k, v = _qkv(gpu, 14, 6, 6, 4, 2, 64, 64, BF)
    f = lambda *s, dtype=BF: torch.randn(*s, device=gpu).to(dtype)  # noqa: E731
    for bad in (dict(k=f(6, 2, 32)), dict(k=f(6, 2, 64, dtype=F)), dict(v=f(5, 2, 64)), dict(v=f(6, 1, 64)), dict(q=f(6, 4, 64, dtype=torch.float16)),
                dict(q=f(1, 6, 4, 64)), dict(cu_seqlens=[0, 6]), dict(cu_seqlens=_i([0, 6], gpu).long()), dict(cu_seqlens=_i([0, 6], gpu), cu_seqlens_k=_i([6], gpu)),
                dict(o=f(6, 4, 32)), dict(o=f(6, 4, 64).half()), dict(q=f(6, 64, 4).transpose(1, 2)), dict(k=None), dict(v=v.cpu()), dict(o_dtype=torch.float16),
                dict(q=f(2, 3, 4, 64), k=f(3, 2, 2, 64), v=f(3, 2, 2, 64))):
        with pytest.raises((ValueError, TypeError)):
            kda.kda_attn_fwd(**{**dict(q=q, k=k, v=v), **bad})
    for bad, word in ((dict(o=q), "ALIAS"), (dict(q=f(6, 3, 64)), "SHAPE"), (dict(cu_seqlens_k=_i([0, 6], gpu)), "NULL"), (dict(scale=math.nan), "SHAPE")):
        with pytest.raises(kda.KdaError, match=word):
            kda.kda_attn_fwd(**{**dict(q=q, k=k, v=v), **bad})
