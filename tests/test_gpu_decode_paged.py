"""kda_decode_step_paged: bit-equal to kda_decode_step on the states of its pages; pages that are out of range or
shared leave the pool and the sequence's row of o alone."""
import pytest
import torch

import kda_inputs as ki
import serving_model as sm

pytestmark = pytest.mark.gpu


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _paged_equals_dense(gpu, tok, pool, ins, outs, o_dtype, z=None, A=None):
    kda = _kda()
    B, H, dv = tok["q"].shape[0], tok["q"].shape[1], tok["v"].shape[-1]
    o = torch.full((B, H, dv), 7.0, device=gpu, dtype=o_dtype)
    got = pool.clone()
    alpha = None if z is not None else tok["alpha"]
    kda.kda_decode_step_paged(tok["q"], tok["k"], tok["v"], alpha, tok["beta"], got, _i(ins, gpu),
                              None if outs is None else _i(outs, gpu), z=z, A=A, o=o)
    outs = ins if outs is None else outs
    want, wo = pool.clone(), torch.full_like(o, 7.0)
    for b, go in enumerate(sm.runs(ins, outs, pool.shape[0])):
        if not go:
            continue
        S = pool[ins[b]:ins[b] + 1].clone()
        one = {n: x[b:b + 1].clone() for n, x in tok.items()}
        if z is None:
            wo[b:b + 1] = kda.kda_decode_step(one["q"], one["k"], one["v"], one["alpha"], one["beta"], S, o_dtype=o_dtype)
        else:
            wo[b:b + 1] = kda.kda_decode_step_gated(one["q"], one["k"], one["v"], z[b:b + 1].clone(), A, one["beta"], S,
                                                    o_dtype=o_dtype)
        want[outs[b]] = S[0]
    torch.cuda.synchronize()
    assert torch.equal(o, wo) and torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_head_sizes(gpu, dtype, dk, dv):
    B, H, P = 5, 3, 9
    tok = ki.make_decode_token(B, H, dk, dv, dtype, seed=dk + dv, device=gpu)
    pool = ki.make_state(P, H, dk, dv, 0.1, 1, gpu)
    _paged_equals_dense(gpu, tok, pool, [8, 0, 3, 5, 1], None, torch.float32)
    _paged_equals_dense(gpu, tok, pool, [8, 0, 3, 5, 1], [8, 2, 4, 6, 1], torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gate(gpu, dtype):
    B, H, P = 6, 4, 7
    tok = ki.make_decode_token(B, H, 128, 64, dtype, seed=3, device=gpu)
    z, A = ki.make_gate((B, H, 128), H, dtype, seed=5, device=gpu)
    pool = ki.make_state(P, H, 128, 64, 0.1, 1, gpu)
    _paged_equals_dense(gpu, tok, pool, [6, 5, 4, 3, -1, 0], None, torch.float32, z=z, A=A)


@pytest.mark.parametrize("ins,outs", [
    ([-1, -1, -1, -1, -1, -1, -1], None),                       # only padding
    ([0, -1, 9, 10, -5, 2 ** 31 - 1, 3], None),                 # out of range
    ([0, 1, 1, 2, 3, 3, 3], None),                              # one page twice, in place
    ([0, 0, 0, 1, 2, 3, 4], [5, 6, 7, 1, 8, 8, 4]),             # forks of one page; two onto one page
    ([0, 0, 1, 2, 3, 4, 5], [0, 6, 2, 3, 7, 8, -1]),            # a parent that runs on in place, a chain
    ([0, 1, 2, 3, 4, 5, 6], [1, 0, 7, 8, 99, -1, 6]),           # a swap
])
def test_pages_that_may_not_run(gpu, ins, outs):
    tok = ki.make_decode_token(7, 2, 64, 32, torch.bfloat16, seed=1, device=gpu)
    pool = ki.make_state(10, 2, 64, 32, 0.1, 2, gpu)
    _paged_equals_dense(gpu, tok, pool, ins, outs, torch.float32)


def test_a_full_call_of_sequences(gpu):
    """4096 sequences, one of which shares its page with the last."""
    kda = _kda()
    B, P = 4096, 5000
    tok = ki.make_decode_token(B, 1, 16, 16, torch.float32, seed=1, device=gpu)
    pool = ki.make_state(P, 1, 16, 16, 0.1, 2, gpu)
    ins = torch.randperm(P, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    ins[17] = ins[-1]
    got = pool.clone()
    o = torch.zeros(B, 1, 16, device=gpu)
    kda.kda_decode_step_paged(tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], got, ins.to(gpu), o=o)
    S = pool[ins.long().to(gpu)].clone()
    wo = kda.kda_decode_step(tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], S)
    runs = torch.ones(B, dtype=torch.bool, device=gpu)
    runs[17] = runs[-1] = False
    want = pool.clone()
    want[ins.long().to(gpu)[runs]] = S[runs]
    assert torch.equal(got, want) and torch.equal(o[runs], wo[runs]) and not o[~runs].any()


def test_far_page(gpu):
    """Pages that start past 2^32 bytes."""
    H, P = 128, 520
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough free memory")
    tok = ki.make_decode_token(1, H, 128, 128, torch.bfloat16, seed=1, device=gpu)
    pool = torch.zeros(P, H, 128, 128, device=gpu)
    assert 4 * (P - 2) * H * 128 * 128 > 2 ** 32
    S = ki.make_state(1, H, 128, 128, 0.1, 2, gpu)
    pool[P - 2] = S[0]
    kda = _kda()
    o = kda.kda_decode_step_paged(tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], pool, _i([P - 2], gpu), _i([P - 1], gpu))
    wo = kda.kda_decode_step(tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], S)
    assert torch.equal(pool[P - 1], S[0]) and torch.equal(o, wo) and not pool[:P - 2].any()
