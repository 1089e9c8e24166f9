"""Prompt attention, of all rows and within a window: scores of any size, and rows that do not see one another's
keys."""
import math

import pytest
import torch

from masked_reference import window_keep

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _rows(n, heads, dim, g, std=1.0):
    return (torch.randn((n, heads, dim), generator=g, device="cuda") * std).to(BF)


def _call(q_, q, k, v, cu, scale, window):
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if window is None:
        return q_.prompt_attention(q, k, v, cu, scale)
    return q_.window_prompt_attention(q, k, v, cu, *window, scale)


# Windows that leave out rows, that no row of the call outgrows, and the call without one.
@pytest.mark.parametrize("window", [None, (100, 3), (399, 0), (400, 0), (1000, 5)])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_of_any_size(q_, dim, window):
    """Scores up to 1e32: the largest visible key has all of the weight, and nothing is lost to the reference."""
    g = torch.Generator(device="cuda").manual_seed(15)
    n = 400
    q, k, v = _rows(n, 2, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    at = torch.arange(n, device="cuda")
    keep = window_keep(at, at, *(window or (n, 0)))
    for size in (1e5, 1e7, 1e9, 1e12, 1e30):
        big = q * size
        out, lse = _call(q_, big, k, v, [0, n], 1.0, window)
        for h in range(2):
            score = torch.where(keep, big[:, h].double() @ k[:, 0].double().T, -math.inf)
            top2 = score.topk(2, 1).values
            # fp32 products and sums: 2^-20 of the magnitudes, and 2^100 between the weights
            near = 2.0 ** -20 * (big[:, h].double().abs() @ k[:, 0].double().abs().T).amax(1)
            clear = top2[:, 0] - top2[:, 1] > 2 * near + 100
            assert clear[1:].float().mean() > 0.9
            assert torch.equal(out[clear, h].double(), v[score.argmax(1)][clear, 0].double())
            assert ((lse[:, h].double() - top2[:, 0]).abs() <= near + 2.0 ** -22 * top2[:, 0].abs() + math.log(n))[clear].all()


@pytest.mark.parametrize("dim", [64, 128])
def test_a_prompt_beside_others_and_alone(q_, dim):
    """Large scores in one sequence of a pack and small ones in the next: the same as alone, and the rows of either
    size in one block."""
    g = torch.Generator(device="cuda").manual_seed(16)
    lens = [300, 500]
    n = sum(lens)
    q, k, v = _rows(n, 2, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    q[100:117] *= 1e9  # in one warp's rows with small ones
    q[::7] *= 1e6
    out, lse = _call(q_, q, k, v, [0, 300, n], 0.1, None)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for rows in (slice(0, 300), slice(300, n)):
        alone, lse2 = _call(q_, q[rows].contiguous(), k[rows].contiguous(), v[rows].contiguous(), [0, rows.stop - rows.start],
                            0.1, None)
        assert torch.equal(out[rows], alone) and torch.equal(lse[rows], lse2)


@pytest.mark.parametrize("window", [None, (150, 3), (500, 0)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [40.0, 1e9, math.nan, math.inf])
def test_a_later_key_changes_no_bit_of_the_rows_before_it(q_, dim, window, size):
    """Nor does one that has left the window: its score moves the reference of rows in the same warp."""
    g = torch.Generator(device="cuda").manual_seed(17)
    n = 900
    q, k, v = _rows(n, 2, dim, g, 1.5), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    clean, lse = _call(q_, q, k, v, [0, n], 0.1, window)
    at = torch.arange(n, device="cuda")
    keep = window_keep(at, at, *(window or (n, 0)))
    for a in (140, 305, 400, 511, 530, 777, 895):
        other = k.clone()
        other[a] *= size
        out, lse2 = _call(q_, q, other, v, [0, n], 0.1, window)
        hit = keep[:, a]
        assert (out[hit] != clean[hit]).any()
        assert torch.equal(lse[~hit], lse2[~hit]) and torch.equal(out[~hit], clean[~hit]), f"key {a}"


@pytest.mark.parametrize("dim", [64, 128])
def test_a_captured_call_within_a_window_follows_the_offsets(q_, dim):
    """A replay takes the offsets that stand there; two graphs of two windows share a workspace in order."""
    g = torch.Generator(device="cuda").manual_seed(18)
    n = 700
    q, k, v = _rows(n, 2, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    cu = torch.tensor([0, 100, n], dtype=torch.int32, device="cuda")
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(n, 2, 1, dim, 2))
    windows, made = ((130, 4), (40, 0)), []
    for window in windows:
        out, lse = torch.empty_like(q), torch.empty((n, 2), device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q_.check(q_.qerl_window_prompt_attention(q, k, v, cu, *window, 0.1, out, lse, ws))
        made.append((graph, out, lse))
    for middle in (100, 0, 511, n):
        cu[1] = middle
        for graph, _, _ in made:
            graph.replay()
        torch.cuda.synchronize()
        for window, (_, out, lse) in zip(windows, made):
            want, lse2 = _call(q_, q, k, v, [0, middle, n], 0.1, window)
            assert torch.equal(out, want) and torch.equal(lse, lse2)
    assert q_.qerl_read_status(ws) == 0
