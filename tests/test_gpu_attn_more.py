"""Calls of the attention layers that the documentation allows: keys and queries turned in place where a page's tokens are read several
times, the largest rotation captured into a graph, bf16 prompts of more than 16K keys."""
import pytest
import torch

from test_gpu_attn_fwd import BF, F, _check, _cu, _i, _kda, _qkv

pytestmark = pytest.mark.gpu
E = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("pairing", ["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 48), (64, 0)])
def test_in_place_on_pages_of_several_fetches(gpu, dtype, cache, pairing, d, rot):
    """On e4m3 pages the rows of a page beyond the first fetch are read for the scale, and again for the codes and the turned rows."""
    kda = _kda()
    lay = kda.KVLayout(cache, 128, 2, d, d)
    before, lens = [0, 100, 5, 127], [300, 200, 1, 129]
    n = sum(lens)
    g = torch.Generator(device=gpu).manual_seed(1)
    row = torch.randn(n, 10, d, generator=g, device=gpu).to(dtype)
    q, k, v = row[:, :6], row[:, 6:8], row[:, 8:]
    table = _i([[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]], gpu)
    freq = 10000.0 ** (-torch.arange(rot // 2, device=gpu).float() / (rot // 2)) if rot else None
    dense, pool = lay.pool(12, gpu), lay.pool(12, gpu)
    for p in (dense, pool):  # (earlier tokens whose codes a larger scale rounds)
        kda.kda_kv_append(row[:127, 6:8].contiguous() / 64, row[:127, 8:].contiguous() / 64, p, lay, table, _i([0], gpu), rows=_i([3], gpu),
                          cu_seqlens=_cu([127], gpu))
    args = (lay, table, _i(before, gpu))
    was, ko = row.clone(), torch.zeros(n, 2, d, dtype=dtype, device=gpu)
    qo, _ = kda.kda_kv_append(k.contiguous(), v.contiguous(), dense, *args, cu_seqlens=_cu(lens, gpu), q=q.contiguous(), inv_freq=freq, pairing=pairing, k_out=ko)
    kda.kda_kv_append(k, v, pool, *args, cu_seqlens=_cu(lens, gpu), q=q, inv_freq=freq, pairing=pairing, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(pool, dense), "pages"
    assert torch.equal(q, qo) and torch.equal(k, ko), "turned rows"
    assert torch.equal(v, was[:, 8:]) and (rot == 0) == torch.equal(row, was)


def test_the_largest_rotation_captured(gpu):
    """Pages of 128 tokens and 128 turned values: more LDS than a kernel has without asking for it."""
    kda = _kda()
    lay = kda.KVLayout(E, 128, 2, 128, 64)
    g = torch.Generator(device=gpu).manual_seed(2)
    k, v = (torch.randn(260, 2, d, generator=g, device=gpu).to(BF) for d in (128, 64))
    freq = 10000.0 ** (-torch.arange(64, device=gpu).float() / 64)
    pool, want, table, lens, cu = lay.pool(4, gpu), lay.pool(4, gpu), _i([[2, 0, 3]], gpu), _i([0], gpu), _cu([260], gpu)
    kda.kda_kv_append(k, v, pool, lay, table, lens, cu_seqlens=cu, inv_freq=freq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_kv_append(k, v, pool, lay, table, lens, cu_seqlens=cu, inv_freq=freq)
    for at in (0, 100, 3):
        lens.fill_(at), k.mul_(-1), pool.zero_(), want.zero_()
        graph.replay()
        kda.kda_kv_append(k, v, want, lay, table, lens, cu_seqlens=cu, inv_freq=freq)
        torch.cuda.synchronize()
        assert torch.equal(pool, want) and pool.any()


@pytest.mark.parametrize("hq,hk,n,m", [(4, 1, 200, 40001), (16, 4, 2000, 20011), (4, 2, 17003, 17003)])
@pytest.mark.parametrize("d", [64, 128])
def test_more_than_16k_keys(gpu, d, hq, hk, n, m):
    q, k, v = _qkv(gpu, 3, n, m, hq, hk, d, d, BF)
    _check(q, k, v, [n], [m], o_dtype=F)
