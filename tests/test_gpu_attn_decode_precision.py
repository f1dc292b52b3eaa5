"""kda_attn_decode with bf16 queries: outputs in fp32 are those of the cached keys and values and of the queries as they are, but
for fp32's own rounding and 2^-16 of the probabilities (two bf16 terms: the first is off by at most 2^-8 of a probability, the
second by 2^-8 of that)."""
import pytest
import torch

import attention_model as am
from test_gpu_attn_decode import BF, E, F, _i, _kda, _model, _pool, _table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [BF, E])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("wide", [False, True])
def test_probabilities_are_not_cut_to_bf16(gpu, cache, dk, dv, K, wide):
    kda = _kda()
    lay, lens = kda.KVLayout(cache, 32, 2, dk, dv), [5, 64, 300, 999]
    P, table = _table([-(-n // 32) for n in lens], gpu, 50, 200 if wide else None)
    pool = _pool(lay, P, gpu, 51)
    q = torch.randn(4, K, 8, dk, generator=torch.Generator(device=gpu).manual_seed(52), device=gpu).to(BF)
    o = kda.kda_attn_decode(q, pool, lay, table.to(gpu), _i(lens, gpu), o_dtype=F)
    args = (lay, pool, table.tolist(), list(range(4)), lens, dk ** -0.5)
    for b, ((ref, cut), (_, exact)) in enumerate(zip(_model(q, *args), _model(q.float(), *args))):
        # (cut - exact is 2^-8 of sum_j p_j |v_j|)
        am.close(o[b], ref, exact + (cut - exact) * 2.0 ** -8, f"sequence {b}")
