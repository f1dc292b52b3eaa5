"""The cosines and sines that kda_kv_append turns by are those of the position times the frequency, rounded to fp32: a pair (1, 0) turns
into (cos, sin) without any other rounding."""
import numpy as np
import pytest
import torch

import attention_model as am

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairing", ["halves", "pairs"])
@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("first", [0, 5000, 1000000])
def test_cosines_and_sines_are_rounded_once(gpu, pairing, rot, first):
    """Within half a step of fp32, and 1e-9 for the product of position and frequency (2^20 / (2 pi) turns and their factor 1 / (2 pi), 2^-53
    each: 4e-10 in the angle) and the series (1.1e-10)."""
    import gated_delta_rule_07_amd as kda
    n, lay = 700, kda.KVLayout(torch.bfloat16, 64, 1, 128, 64)
    pos = list(range(first, first + n - 3)) + [-1, -first - 77, 1]
    freq = 10000.0 ** (-torch.arange(rot // 2, device=gpu).float() / (rot // 2))
    freq[1::3] *= -1.7  # (any frequency)
    a, b = (torch.arange(rot // 2), torch.arange(rot // 2) + rot // 2) if pairing == "halves" else (2 * torch.arange(rot // 2), 2 * torch.arange(rot // 2) + 1)
    q = torch.zeros(n, 1, 128, device=gpu)
    q[..., a] = 1.0
    cu, table = torch.tensor([0, n], dtype=torch.int32, device=gpu), torch.zeros(1, 1, dtype=torch.int32, device=gpu)
    k = q.clone()
    ko = torch.zeros_like(q)
    qo, _ = kda.kda_kv_append(k, q[..., :64].contiguous(), lay.pool(1, gpu), lay, table, torch.zeros(1, dtype=torch.int32, device=gpu), cu_seqlens=cu, q=q,
                              inv_freq=freq, positions=torch.tensor(pos, dtype=torch.int32, device=gpu), pairing=pairing, k_out=ko)
    angle = np.array(pos, dtype=np.longdouble)[:, None] * freq.cpu().numpy().astype(np.longdouble)
    for out in (qo, ko):
        for got, want in ((out[:, 0, a], np.cos(angle)), (out[:, 0, b], np.sin(angle))):
            off = np.abs(got.cpu().numpy().astype(np.longdouble) - want)
            over = off - (am.U * np.abs(want) + 1e-9)
            assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.size}, worst {float((off / (am.U * np.abs(want) + 1e-9)).max()):.3g} of the bound"
