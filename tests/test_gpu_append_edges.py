"""The append at its edges: a cache without pages."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _no_freq():
    return torch.empty(0, dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F8])
def test_a_cache_without_pages_records_the_lost_tokens(q_, dtype):
    none = torch.empty((0, 2, 16, 64), dtype=dtype, device="cuda")
    cache = q_.kv_cache(none, none, torch.zeros((3, 4), dtype=torch.int32, device="cuda"))
    k = torch.randn((3, 2, 64), device="cuda").to(BF)
    k_out = torch.zeros_like(k)
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_rope_append(cache, None, k, k, pos, _no_freq(), None, k_out, ws))
    assert q_.STATUS_NAMES[q_.qerl_read_status(ws)] == "QERL_ERR_RANGE"
    assert torch.equal(k_out, k)  # the rotation (here by nothing) is done all the same
    # padding needs no place
    q_.check(q_.qerl_rope_append(cache, None, k, k, pos - 1, _no_freq(), None, k_out, ws))
    assert q_.qerl_read_status(ws) == 0
    # attention over it finds no page either
    dws = q_.workspace(q_.qerl_decode_attention_workspace_size(3, 4, 2, 64))
    q = torch.randn((3, 4, 64), device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    q_.check(q_.qerl_decode_attention(cache, q, pos + 5, 0.1, out, lse, dws))
    assert q_.STATUS_NAMES[q_.qerl_read_status(dws)] == "QERL_ERR_RANGE"
    assert (out == 0).all()
