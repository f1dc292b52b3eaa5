"""Outputs that a serving call makes itself hold nothing of what their memory held before: zeros in the rows that the call
passes over, pairs of -1 behind a move list."""
import pytest
import torch

import kda_inputs as ki

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _kda():
    import gated_delta_rule_07_amd as kda
    return kda


def _i(x, gpu):
    return torch.tensor(x, dtype=torch.int32, device=gpu)


def _spoil(gpu, *sizes):
    """The allocator's next blocks of these sizes (in floats) hold NaN."""
    blocks = [torch.full((n,), NAN, device=gpu) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("o_dtype", [torch.float32, torch.bfloat16])
def test_decode_rows_passed_over(gpu, side, o_dtype):
    kda = _kda()
    B, H, d = 6, 3, 64
    tok = ki.make_decode_token(B, H, d, d, torch.bfloat16, seed=1, device=gpu)
    pool = ki.make_state(9, H, d, d, 0.1, 2, gpu)
    ins = _i([4, -1, 7, 9, 2, 2], gpu)  # padding, out of range, one page twice
    want = torch.zeros(B, H, d, device=gpu, dtype=o_dtype)
    kda.kda_decode_step_paged(*(tok[n] for n in ("q", "k", "v", "alpha", "beta")), pool.clone(), ins, o=want)
    _spoil(gpu, want.numel() * want.element_size() // 4)
    stream = None
    if side:  # (the fill belongs to the call's stream: the current one is still busy when the call runs)
        stream = torch.cuda.Stream()
        torch.cuda._sleep(20_000_000)
    o = kda.kda_decode_step_paged(*(tok[n] for n in ("q", "k", "v", "alpha", "beta")), pool, ins, o_dtype=o_dtype, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and want[0].any() and want[2].any() and not want[[1, 3, 4, 5]].any()


@pytest.mark.parametrize("side", [False, True])
def test_tree_rows_passed_over(gpu, side):
    kda = _kda()
    B, K, H, d = 3, 5, 2, 32
    x = ki.make_prefill(B, K, H, d, d, torch.float32, 3.0, 0.1, seed=4, device=gpu)
    args = [x[n] for n in ("q", "k", "v", "alpha", "beta")]
    pool, par = ki.make_state(4, H, d, d, 0.1, 5, gpu), _i([[-1, 0, 0, 1, 3]] * B, gpu)
    for pages, nodes in ((_i([3, -1, 0], gpu), None), (None, _i([5, 0, 2], gpu)), (_i([1, 4, 2], gpu), _i([3, 5, 5], gpu))):
        wo, wu = torch.zeros(B, K, H, d, device=gpu), torch.zeros(B, H, K, d, device=gpu)
        kda.kda_tree_verify(*args, pool, pages, par, nodes, o=wo, u=wu)
        _spoil(gpu, wo.numel())
        stream = torch.cuda.Stream() if side else None
        if side:
            torch.cuda._sleep(20_000_000)
        o, u = kda.kda_tree_verify(*args, pool, pages, par, nodes, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(u, wu)
        assert wo[0].any() and not wo[1, 3:].any()


def test_outputs_made_inside_a_capture(gpu):
    """A captured call's own outputs are filled by the graph, on every replay."""
    kda = _kda()
    B, H, d = 4, 2, 32
    tok = ki.make_decode_token(B, H, d, d, torch.float32, seed=1, device=gpu)
    pool = ki.make_state(6, H, d, d, 0.1, 2, gpu)
    other, pages = pool.clone(), _i([0, 1, 2, 3], gpu)
    args = [tok[n] for n in ("q", "k", "v", "alpha", "beta")]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = kda.kda_decode_step_paged(*args, pool, pages)
    for turn in ([0, 1, 2, 3], [5, -1, 5, 4], [-1, 0, 6, 1]):
        pages.copy_(_i(turn, gpu))
        graph.replay()
        want = torch.zeros(B, H, d, device=gpu)
        kda.kda_decode_step_paged(*args, other, pages, o=want)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(pool, other)


@pytest.mark.parametrize("side", [False, True])
def test_move_lists_hold_nothing_behind_their_moves(gpu, side):
    """A list used whole, without its count, moves what it should and nothing else."""
    kda = _kda()
    table, ref = _i([[0], [-1], [-1], [-1], [-1]], gpu), _i([1, 0, 0], gpu)
    parents, children = _i([0, 0, 0, 0], gpu), _i([1, 2, 3, 4], gpu)
    old = [_i([[0, 1], [0, 2], [1, 0], [2, 1]] * 4, gpu) for _ in range(8)]  # (what the next list's memory held)
    torch.cuda.synchronize()
    del old
    stream = torch.cuda.Stream() if side else None
    if side:
        torch.cuda._sleep(20_000_000)
    moves, n = kda.kda_cache_fork(table, ref, parents, children, stream=stream)
    torch.cuda.synchronize()
    assert moves[:2].tolist() == [[0, 1], [0, 2]]
    assert int(n) == 2 and moves[2:].tolist() == [[-1, -1]] * 2
    pool = torch.arange(3.0, device=gpu).view(3, 1).expand(3, 4).contiguous()
    kda.kda_cache_copy(pool, moves)
    assert pool[:, 0].tolist() == [0.0, 0.0, 0.0]
    kda.kda_cache_free(table, ref, _i([0], gpu))
    t2, r2, moves, n, live = kda.kda_cache_compact(table, ref, stream=stream)
    torch.cuda.synchronize()
    assert int(live) == 2 and int(n) == 1 and moves.tolist() == [[2, 0]]
