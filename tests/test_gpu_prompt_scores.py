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
