"""Tensors that a call makes itself -- outputs that are not given, workspaces -- are memory of the call's stream.  A block of
another stream's memory may still be in use there, and may be handed out there again as soon as its tensor is gone, with nothing
that orders either against the call.

The calls run here on the CPU with the library and the checks of devices taken out: what is looked at is where the tensors are made."""
import contextlib

import pytest
import torch

BF, F, I = torch.bfloat16, torch.float32, torch.int32


class _Stream:
    cuda_stream = 1


STREAM = _Stream()


class _Lib:
    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def made(monkeypatch):
    """(module, list of the streams on which tensors were made)."""
    import gated_delta_rule_07_amd as kda
    on, streams = [None], []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def noted(fn):
        def call(*a, **kw):
            streams.append(on[-1])
            return fn(*a, **kw)
        return call

    monkeypatch.setattr(kda, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(kda, "_device_of", lambda t, name: 0)
    monkeypatch.setattr(kda, "_need", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(kda, "_rows", lambda *a: None)
    monkeypatch.setattr(kda, "_check", lambda *a: None)
    monkeypatch.setattr(kda, "_run", lambda *a: None)
    monkeypatch.setattr(kda, "_stream", lambda *a: None)
    monkeypatch.setattr(kda, "load_library", lambda: _Lib())
    monkeypatch.setattr(kda, "kda_chunk_fwd_split_plan", lambda *a, **kw: (4, 256))
    monkeypatch.setattr(kda, "kda_attn_decode_plan", lambda *a: 256)
    monkeypatch.setattr(kda, "_page_bytes", lambda dtype, pt, H, dk, dv: H * pt * (dk + dv) * 2)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "full", "zeros", "empty_like", "full_like", "zeros_like"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    return kda, streams


def _calls():
    t = lambda *s: torch.ones(*s, dtype=BF)  # noqa: E731
    f = lambda *s: torch.ones(*s)  # noqa: E731
    i = lambda *s: torch.ones(*s, dtype=I)  # noqa: E731
    x4, a4, b4 = t(1, 5, 2, 64), f(1, 5, 2, 64), f(1, 5, 2)
    x3, a3, b3, S = t(3, 2, 64), f(3, 2, 64), f(3, 2), f(3, 2, 64, 64)
    lay = lambda k: k.KVLayout(BF, 16, 2, 64, 64)  # noqa: E731
    pool = torch.ones(4, 2 * 16 * 128 * 2, dtype=torch.uint8)
    # name: (call, tensors it makes)
    return {
        "chunk": (lambda k, s: k.kda_chunk_fwd(x4, x4, x4, a4, b4, stream=s), 2),
        "snapshots": (lambda k, s: k.kda_chunk_fwd_snapshots(x4, x4, x4, a4, b4, snap_tokens=[5], stream=s), 3),
        "varlen": (lambda k, s: k.kda_chunk_fwd_varlen(x3, x3, x3, a3, b3, i(3), stream=s), 2),
        "gated": (lambda k, s: k.kda_chunk_fwd_gated(x4, x4, x4, x4, f(2), b4, stream=s), 2),
        "split": (lambda k, s: k.kda_chunk_fwd_split(x4, x4, x4, a4, b4, stream=s), 3),
        "split_noalloc": (lambda k, s: k.kda_chunk_fwd_split_noalloc(x4, x4, x4, a4, b4, stream=s), 2),
        "step": (lambda k, s: k.kda_decode_step(x3, x3, x3, a3, b3, S, stream=s), 1),
        "step_gated": (lambda k, s: k.kda_decode_step_gated(x3, x3, x3, x3, f(2), b3, S, stream=s), 1),
        "verify": (lambda k, s: k.kda_decode_verify(x4, x4, x4, a4, b4, f(1, 2, 64, 64), stream=s), 2),
        "qk_norm": (lambda k, s: k.kda_qk_norm(x3, x3, stream=s), 2),
        "fork": (lambda k, s: k.kda_cache_fork(i(2, 3), i(4), i(1), i(1), stream=s), 2),
        "compact": (lambda k, s: k.kda_cache_compact(i(2, 3), i(4), stream=s), 5),
        "step_paged": (lambda k, s: k.kda_decode_step_paged(x3, x3, x3, a3, b3, f(4, 2, 64, 64), i(3), stream=s), 1),
        "tree": (lambda k, s: k.kda_tree_verify(x4, x4, x4, a4, b4, f(4, 2, 64, 64), i(1), i(1, 5), stream=s), 2),
        "attn_fwd": (lambda k, s: k.kda_attn_fwd(x3, x3, x3, stream=s), 1),
        "attn_fwd_packed": (lambda k, s: k.kda_attn_fwd(x3, x3, x3, cu_seqlens=i(2), stream=s), 1),
        "append": (lambda k, s: k.kda_kv_append(x3, x3, pool, lay(k), i(3, 1), i(3), q=x3, stream=s), 1),
        "append_packed": (lambda k, s: k.kda_kv_append(x3, x3, pool, lay(k), i(3, 1), i(1), q=x3, cu_seqlens=i(2), stream=s), 1),
        "read": (lambda k, s: k.kda_kv_read(pool, lay(k), i(3, 1), i(2), 5, stream=s), 2),
        "decode": (lambda k, s: k.kda_attn_decode(x3, pool, lay(k), i(3, 1), i(3), stream=s), 2),
        "decode_rows": (lambda k, s: k.kda_attn_decode(x3, pool, lay(k), i(3, 1), i(3), rows=i(3), stream=s), 2),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_made_on_the_calls_stream(made, name):
    kda, streams = made
    call, n = _calls()[name]
    streams.clear()
    call(kda, STREAM)
    assert streams == [STREAM] * n
    kda._raw_stream = lambda index: 1  # (the current one: nothing to change)
    streams.clear()
    call(kda, STREAM)
    assert streams == [None] * n
    streams.clear()
    call(kda, None)
    assert streams == [None] * n


@pytest.mark.gpu
def test_blocks_of_another_stream_are_not_taken(gpu):
    """A block that the current stream's work has just dropped is not where a call on another stream writes."""
    import gated_delta_rule_07_amd as kda
    n, H, d = 300, 4, 128
    g = torch.Generator(device=gpu).manual_seed(1)
    x = torch.randn(n, H, d, generator=g, device=gpu).to(BF)
    lay = kda.KVLayout(BF, 64, H, d, d)
    pool, lens = lay.pool(5, gpu), torch.zeros(1, dtype=I, device=gpu)
    full = torch.full((1,), n, dtype=I, device=gpu)
    table, cu = torch.arange(5, dtype=I, device=gpu)[None], torch.tensor([0, n], dtype=I, device=gpu)
    side = torch.cuda.Stream()

    def calls(stream):
        o = kda.kda_attn_fwd(x, x, x, cu_seqlens=cu, stream=stream)
        turned, _ = kda.kda_kv_append(x, x, pool, lay, table, lens, cu_seqlens=cu, q=x, stream=stream)
        k, v = kda.kda_kv_read(pool, lay, table, cu, n, stream=stream)
        last = kda.kda_attn_decode(x[:1], pool, lay, table, full, stream=stream)
        return [o, turned, k, v, last]

    want = calls(None)
    torch.cuda.synchronize()
    dropped = [torch.empty_like(t) for t in want for _ in range(4)]
    blocks = {t.data_ptr() for t in dropped}
    del dropped
    torch.cuda.synchronize()
    got = calls(side)
    torch.cuda.synchronize()
    assert not blocks & {t.data_ptr() for t in got}
    assert all(torch.equal(a, b) for a, b in zip(got, want))
