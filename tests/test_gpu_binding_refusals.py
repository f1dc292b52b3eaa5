"""Arguments of the serving calls that do not belong together, or are no tensors, are refused in words, with the compiled
argument helper and without it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[True, False], ids=["helper", "python"])
def kda(request, gpu, monkeypatch):
    import gated_delta_rule_07_amd as kda
    if not request.param:
        monkeypatch.setattr(kda, "_need", kda._need_in_words)
        monkeypatch.setattr(kda, "_rows", lambda t, dtype, index: None)
    return kda


def test_norms_of_tokens_that_do_not_match(gpu, kda):
    """As many keys as queries is not enough: batch and token counts agree, and so do those of [B,T] positions."""
    f = lambda *s: torch.randn(*s, device=gpu)  # noqa: E731
    q, freq = f(2, 3, 4, 32), f(8)
    pos = torch.arange(6, dtype=torch.int32, device=gpu)
    for bad in (dict(k=f(3, 2, 4, 32)), dict(k=f(6, 1, 4, 32)), dict(k=f(6, 4, 32)), dict(inv_freq=freq, positions=pos.view(3, 2)),
                dict(inv_freq=freq, positions=pos.view(1, 6)), dict(inv_freq=freq, positions=pos[:5])):
        with pytest.raises(ValueError, match="agree|one entry per token"):
            kda.kda_qk_norm(q, **bad)
    want = kda.kda_qk_norm(q.view(6, 4, 32), inv_freq=freq, positions=pos)[0]
    for good in (pos, pos.view(2, 3)):
        assert torch.equal(kda.kda_qk_norm(q, f(2, 3, 2, 32), inv_freq=freq, positions=good)[0].view(6, 4, 32), want)
    assert torch.equal(kda.kda_qk_norm(q.view(6, 4, 32), inv_freq=freq, positions=pos.view(3, 2))[0], want)


def test_what_is_no_tensor(gpu, kda):
    f = lambda *s: torch.randn(*s, device=gpu)  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    q, freq = f(6, 4, 32), f(8)
    table, ref, one = i([0], [-1]), i(1, 0), i(1)
    tok, pool = [f(1, 2, 16) for _ in range(4)] + [f(1, 2)], f(2, 2, 16, 16)
    tree = [f(1, 3, 2, 16) for _ in range(4)] + [f(1, 3, 2)]
    for call in (lambda: kda.kda_qk_norm(q, inv_freq=[0.5] * 8, positions=i(0, 1, 2, 3, 4, 5)), lambda: kda.kda_qk_norm(q, [1]),
                 lambda: kda.kda_qk_norm(q, inv_freq=freq, positions=[0, 1, 2, 3, 4, 5]), lambda: kda.kda_qk_norm(q, q_out=[0]),
                 lambda: kda.kda_qk_norm(q, q_weight=[1.0] * 32), lambda: kda.kda_qk_norm(q, q.clone(), k_out=3),
                 lambda: kda.kda_cache_fork(table, ref, [0], one), lambda: kda.kda_cache_fork(table, ref, i(0), one, moves=[[0, 0]]),
                 lambda: kda.kda_cache_fork(table, ref, i(0), one, n_moves=1), lambda: kda.kda_cache_free(table, ref, [0]),
                 lambda: kda.kda_cache_compact(table, ref, moves=0), lambda: kda.kda_cache_copy(pool, [[0, 1]]),
                 lambda: kda.kda_decode_step_paged(*tok, pool, [0]), lambda: kda.kda_decode_step_paged(*tok, pool, i(0), o=0),
                 lambda: kda.kda_tree_verify(*tree, pool, i(0), [-1, 0, 1]), lambda: kda.kda_tree_verify(*tree, pool, i(0), i([-1, 0, 1]), o=[]),
                 lambda: kda.kda_tree_verify(*tree, pool, i(0), i([-1, 0, 1]), u=1)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()
    with pytest.raises(ValueError, match="moves"):
        kda.kda_cache_fork(table, ref, i(0), one, moves=i(0, 1))
    with pytest.raises(ValueError, match="moves"):
        kda.kda_cache_fork(table, ref, i(0), one, moves=torch.tensor(3, dtype=torch.int32, device=gpu))
    assert table.tolist() == [[0], [-1]] and ref.tolist() == [1, 0]
