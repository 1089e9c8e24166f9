"""Prompt attention at the ends of its documented range: the longest sequence, offsets that break their
order, a million sequences."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _call(q_, q, k, v, cu, scale):
    t, h, d = q.shape
    out, lse = torch.full_like(q, 5.0), torch.full((t, h), 5.0, device="cuda")
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(t, h, k.shape[1], d, cu.numel() - 1))
    q_.check(q_.qerl_prompt_attention(q, k, v, cu, scale, out, lse, ws))
    return out, lse, q_.STATUS_NAMES[q_.qerl_read_status(ws)]


def _cu(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def test_a_sequence_longer_than_the_limit_is_recorded_and_skipped(q_):
    t = 2 ** 24 + 1
    x = torch.zeros((t, 1, 64), dtype=BF, device="cuda")
    out, lse, status = _call(q_, x, x, x, _cu([0, t]), 0.1)
    assert status == "QERL_ERR_RANGE"
    assert (out == 5).all() and (lse == 5).all()
    # a call may have more rows than that
    out, lse, status = _call(q_, x, x, x, _cu([0, 1, 300]), 0.1)
    assert status == "QERL_OK"
    assert (out[:300] == 0).all() and (out[300:] == 5).all() and (lse[300:] == 5).all()


@pytest.mark.parametrize("offsets", [[0, 60, 40, 100], [0, 100, 0, 100], [0, 50, 101], [-1, 50, 100], [10, 5, 20, 100]])
def test_broken_offsets_leave_every_row_alone(q_, offsets):
    """Sequences around a step back would overlap: rows of two sequences at once have no right value."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((100, h, 64), generator=g, device="cuda").to(BF) for h in (2, 1, 1))
    out, lse, status = _call(q_, q, k, v, _cu(offsets), 0.1)
    assert status == "QERL_ERR_RANGE"
    assert (out == 5).all() and (lse == 5).all()
    out, lse, status = _call(q_, q, k, v, _cu([0, 60, 60, 100]), 0.1)
    assert status == "QERL_OK" and (out != 5).any(-1).all() and (lse != 5).all()
