"""kda_attn_decode with more sequences than a workgroup has threads, shared out among the workgroups: a thread then sums and writes
the granules of several sequences, and borders of the workgroups' runs fall inside sequences of all kinds."""
import pytest
import torch

import attention_model as am
from test_gpu_attn_decode import BF, E, F, _i, _kda, _model, _pool, _table

pytestmark = pytest.mark.gpu


def _lens(B):
    """Short ones, empty ones, and some long ones, among them neighbours and the last one."""
    lens = [(37 * b * b + 11 * b) % 190 if b % 5 else 0 for b in range(B)]
    for b, n in ((0, 2500), (1, 4100), (B // 3, 1), (B // 2, 3333), (B // 2 + 1, 129), (B - 2, 0), (B - 1, 4999)):
        lens[b] = n
    return lens


@pytest.mark.parametrize("B", [255, 256, 257, 511, 1000])
@pytest.mark.parametrize("cache,dtype,K,hq,hk", [(E, BF, 1, 4, 1), (BF, BF, 2, 4, 2), (E, F, 1, 20, 1)])
def test_more_sequences_than_threads(gpu, B, cache, dtype, K, hq, hk):
    kda = _kda()
    lay, lens = kda.KVLayout(cache, 16, hk, 64, 64), _lens(B)
    P, table = _table([-(-n // 16) for n in lens], gpu, 60, 320)  # 5,120 tokens a row
    pool = _pool(lay, P, gpu, 61)
    rows = [-1 if b % 7 == 3 and b not in (0, 1, B // 2, B - 1) else b for b in range(B)]
    q = torch.randn(B, K, hq, 64, generator=torch.Generator(device=gpu).manual_seed(62), device=gpu).to(dtype)
    assert kda.kda_attn_decode_plan(lay, B, K, hq, table.shape[1]) > 0, "units taken whole"
    o = torch.full((B, K, hq, 64), 7.0, device=gpu, dtype=dtype)
    kda.kda_attn_decode(q, pool, lay, table.to(gpu), _i(lens, gpu), rows=_i(rows, gpu), o=o)
    for b, want in enumerate(_model(q, lay, pool, table.tolist(), rows, lens, 0.125)):
        if want is None:
            assert bool((o[b] == 7).all()), f"sequence {b}: padding"
        else:
            am.close(o[b], *want, what=f"sequence {b} of {lens[b]}")


def test_as_many_as_a_call_takes(gpu):
    """4,096 sequences, shared out: 16 for each thread."""
    kda = _kda()
    B, lay = 4096, kda.KVLayout(E, 128, 1, 64, 128)
    lens = [0] * B
    for b, n in ((0, 5), (1, 4500), (15, 128), (16, 300), (700, 17), (2047, 129), (2048, 1), (4000, 4090), (4094, 2), (4095, 5000)):
        lens[b] = n
    rows = [b if lens[b] or b % 3 else -1 for b in range(B)]
    P, table = _table([-(-n // 128) for n in lens], gpu, 63, 40)
    pool = _pool(lay, P, gpu, 64)
    q = torch.randn(B, 2, 64, generator=torch.Generator(device=gpu).manual_seed(65), device=gpu).to(BF)
    assert kda.kda_attn_decode_plan(lay, B, 1, 2, 40) > 0, "units taken whole"
    o = torch.full((B, 2, 128), 7.0, device=gpu, dtype=BF)
    kda.kda_attn_decode(q, pool, lay, table.to(gpu), _i(lens, gpu), rows=_i(rows, gpu), o=o)
    some = [b for b in range(B) if lens[b]]
    for b, want in zip(some, _model(q[some][:, None], lay, pool, table.tolist(), some, [lens[b] for b in some], 0.125)):
        am.close(o[b:b + 1], *want, what=f"sequence {b} of {lens[b]}")
    none = torch.tensor([r < 0 for r in rows], device=gpu)
    empty = torch.tensor([r >= 0 and not n for r, n in zip(rows, lens)], device=gpu)
    assert bool((o[none] == 7).all()) and not o[empty].any()
