"""Prompt attention at the ends of its documented range: the longest sequence, offsets that break their
order, a million sequences."""
import pytest
import torch

from attention_reference import assert_within, attend64

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


@pytest.mark.parametrize("n,at,long", [(5000, 1700, 2000), (2 ** 20, 700001, 100000), (2 ** 20, 2 ** 20 - 1, 300)])
def test_a_long_sequence_among_many_short_ones(q_, n, at, long):
    """Up to the documented number of sequences, of no or one row but for one: every row is right, and finding
    the blocks does not take long (looking at all sequences for each block of the long one takes seconds)."""
    g = torch.Generator(device="cuda").manual_seed(n + at)
    lens = torch.randint(0, 2, (n,), generator=g, device="cuda")
    lens[at] = long
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    t, begin = int(cu[-1]), int(cu[at])
    q, k, v = (torch.randn((t, 1, 64), generator=g, device="cuda").to(BF) for _ in range(3))
    _call(q_, q, k, v, cu, 0.125)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, lse, status = _call(q_, q, k, v, cu, 0.125)
    end.record()
    torch.cuda.synchronize()
    assert status == "QERL_OK" and start.elapsed_time(end) < 1000
    one = torch.ones(t, dtype=torch.bool, device="cuda")
    one[begin:begin + long] = False
    # a row alone attends to itself: the score to fp32's 2^-20 of its products' magnitudes
    near = 2.0 ** -20 * (1 + 0.125 * (q.double() * k.double()).abs().sum(-1))
    assert torch.equal(out[one], v[one])
    want = 0.125 * (q.double() * k.double()).sum(-1)
    assert ((lse.double() - want).abs() <= near + 2.0 ** -22 * want.abs())[one].all()
    for i in (0, 255, 256, long // 2, long - 1):
        rows = slice(begin, begin + i + 1)
        o, l, to, tl = attend64(q[begin + i], k[rows, 0], v[rows, 0], 0.125, "bf16")
        assert_within(out[begin + i], o, to, f"row {i}")
        assert_within(lse[begin + i], l, tl, f"lse of row {i}")
