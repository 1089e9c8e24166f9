"""Attention of one new token over an E4M3 cache at scores whose fp32 steps are as large as the range that a weight
may pass the running reference by."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("heads,dim", [(4, 64), (12, 64), (4, 128), (12, 128)])
@pytest.mark.parametrize("window", [None, (700, 5)])
@pytest.mark.parametrize("bits", [24, 25, 26, 27, 28, 30])
def test_a_key_one_step_above_the_others(heads, dim, window, bits):
    """Scores (base 2) of 1.0078125 * 2^bits, and of a few steps of fp32 more at every 97th key, from 16 on: all of
    the weight (but for 2^-16 of it) is theirs, and the output their value."""
    import nvfp4_weight_quantized_03_gb300 as q_
    n, seqs, page = 900, 400, 32
    step = max(16.0, 2.0 ** (bits - 23))
    k, v = torch.zeros((1, 928, dim), device="cuda"), torch.ones((1, 928, dim), device="cuda")
    k[:, :, 0] = 1.0
    k[:, 400::97, 1] = 1.0
    v[:, 400::97] = 0.5
    pages = [x.to(F8).view(torch.uint8).view(1, 29, page, dim).transpose(0, 1).contiguous().view(F8) for x in (k, v)]
    table = torch.arange(29, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    q = torch.zeros((seqs, heads, dim), dtype=BF, device="cuda")
    q[:, :, 0], q[:, :, 1] = 2.0 ** bits * 1.0078125, step
    scale = float(torch.tensor(2.0, dtype=torch.float64).log())
    lengths = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    cache = q_.kv_cache(*pages, table)
    out, _ = q_.decode_attention(cache, q, lengths, scale) if window is None else \
        q_.window_decode_attention(cache, q, lengths, *window, scale)
    # 6 keys of 900 at 2^16 and more of the others' weight: the others have 900 / 6 * 2^-16 = 0.0023 of the sum at
    # most, their values are 0.5 larger, and the output is rounded to bf16 (2^-9 at 0.5)
    assert torch.isfinite(out.float()).all()
    assert ((out.double() - 0.5).abs() <= 0.0023 * 0.5 + 2.0 ** -9).all()
