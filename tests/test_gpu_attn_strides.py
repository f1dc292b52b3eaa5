"""kda_attn_fwd on bf16 keys and values whose rows lie so far apart that 64 of them take up to 2^31 bytes, and farther: on both sides
of the border between the kernels that copy tiles by 32-bit offsets and those that do not."""
import pytest
import torch

import attention_model as am
from test_gpu_attn_fwd import BF, F, _cu, _kda

pytestmark = pytest.mark.gpu
BORDER = 1 << 24  # elements between rows


def _far(gpu, m, stride, hk, dk, dv, seed):
    """Keys and values of m tokens in rows `stride` elements apart."""
    if torch.cuda.mem_get_info()[0] < 2 * m * stride + (8 << 30):
        pytest.skip("not enough free memory")
    g = torch.Generator(device=gpu).manual_seed(seed)
    buf = torch.empty(m, stride, dtype=BF, device=gpu)
    k, v = (buf[:, a:a + hk * d].unflatten(1, (hk, d)) for a, d in ((0, dk), (stride - hk * dv, dv)))
    for x in (k, v):
        x.copy_(torch.randn(x.shape, generator=g, device=gpu))
    return k, v


def _check(gpu, n, lens_k, k, v, hq, seed):
    q = torch.randn(n, hq, k.shape[2], generator=torch.Generator(device=gpu).manual_seed(seed), device=gpu).to(BF)
    o = torch.full((n, hq, v.shape[2]), 7.0, device=gpu)
    _kda().kda_attn_fwd(q, k, v, cu_seqlens=_cu([n], gpu), cu_seqlens_k=_cu(lens_k, gpu), o=o)
    ref, slack = am.fwd(q, k.contiguous(), v.contiguous(), k.shape[2] ** -0.5, [n], lens_k)
    am.close(o, ref, slack, "o")
    near = torch.empty_like(o)
    _kda().kda_attn_fwd(q, k.contiguous(), v.contiguous(), cu_seqlens=_cu([n], gpu), cu_seqlens_k=_cu(lens_k, gpu), o=near)
    return o, near


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("hq,hk", [(4, 2), (258, 2)])
def test_just_below_the_border(gpu, dk, dv, hq, hk):
    """The waves of a workgroup share the keys (few heads), or the queries (many): the same kernels as for rows side by side."""
    k, v = _far(gpu, 70, BORDER - 8, hk, dk, dv, 1)
    o, near = _check(gpu, 70, [70], k, v, hq, 2)
    assert torch.equal(o, near)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("stride", [BORDER, BORDER + 8])
def test_from_the_border_on(gpu, dk, dv, stride):
    k, v = _far(gpu, 70, stride, 2, dk, dv, 3)
    _check(gpu, 70, [70], k, v, 4, 4)
    _check(gpu, 33, [70], k, v, 6, 5)


def test_one_of_the_two_strides(gpu):
    k, v = _far(gpu, 40, BORDER, 2, 64, 128, 6)
    _check(gpu, 40, [40], k.contiguous(), v, 4, 7)
    _check(gpu, 40, [40], k, v.contiguous(), 4, 8)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_long_enough_for_32_queries_a_workgroup(gpu, dk, dv):
    k, v = _far(gpu, 520, BORDER, 2, dk, dv, 9)
    _check(gpu, 520, [520], k, v, 16, 10)
