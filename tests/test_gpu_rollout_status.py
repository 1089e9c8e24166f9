"""The rollout example reports what the device recorded in any of its passes."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_status_of_every_pass():
    import nvfp4_weight_quantized_03_gb300 as q
    from rollout_block import AttentionHalf
    half = AttentionHalf(8, 2, 64, 2, 40)
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn((50, half.hidden), generator=g, device="cuda").to(torch.bfloat16)
    half.prompts(h, [30, 20])
    assert half.status() == q.QERL_OK
    half.prompts(h, [49, 1])  # three pages of 16 rows do not take the first
    assert q.STATUS_NAMES[half.status()] == "QERL_ERR_RANGE" and half.status() == q.QERL_OK
    half.prompts(h, [30, 20])
    x = h[:, :8 * 64].unflatten(1, (8, 64)).contiguous()
    back = torch.tensor([0, 30, 20], dtype=torch.int32, device="cuda")
    q.check(q.qerl_prompt_attention(x, x, x, back, 0.1, torch.empty_like(x), None, half.prompt_ws[-1]))
    assert q.STATUS_NAMES[half.status()] == "QERL_ERR_RANGE" and half.status() == q.QERL_OK


def test_one_workspace_for_the_three_calls():
    """They write only the status word of it, or leave it as it was: they take turns on one."""
    import nvfp4_weight_quantized_03_gb300 as q
    heads, kv_heads, dim, page, lens = 8, 2, 64, 16, [37, 20]
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda n, h: torch.randn((n, h, dim), generator=g, device="cuda").to(torch.bfloat16)
    pages = [torch.zeros((6, kv_heads, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = q.kv_cache(*pages, torch.tensor([[4, 0, 3], [2, 5, 1]], dtype=torch.int32, device="cuda"))
    freq = torch.linspace(1, 0.01, dim // 2, dtype=torch.float64, device="cuda")
    tokens = sum(lens)
    ws = q.workspace(max(q.qerl_rope_append_workspace_size(),
                         q.qerl_decode_attention_workspace_size(2, heads, kv_heads, dim),
                         q.qerl_prompt_attention_workspace_size(tokens, heads, kv_heads, dim, 2)))
    positions = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
    seq_ids = torch.repeat_interleave(torch.arange(2, dtype=torch.int32), torch.tensor(lens)).cuda()
    cu = torch.tensor([0, 37, 57], dtype=torch.int32, device="cuda")
    vh = rnd(tokens, kv_heads)
    qr, kr = q.rope_append(cache, rnd(tokens, heads), rnd(tokens, kv_heads), vh, positions, freq, seq_ids, ws=ws)
    whole, _ = q.prompt_attention(qr, kr, vh, cu, dim ** -0.5, ws=ws)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    last, _ = q.decode_attention(cache, qr[[36, 56]], lengths, dim ** -0.5, ws=ws)  # the prompts' last rows again
    # both round to bf16 (2^-8 each), the prompt's weights too; |v| < 6 and the weights sum to 1
    assert ((last.double() - whole[[36, 56]].double()).abs() < 6 * 3 * 2.0 ** -8).all()
    assert q.qerl_read_status(ws) == q.QERL_OK
    # a token where the table has no column
    q.rope_append(cache, rnd(2, heads), rnd(2, kv_heads), rnd(2, kv_heads), lengths + 20, freq, ws=ws)
    assert q.STATUS_NAMES[q.qerl_read_status(ws)] == "QERL_ERR_RANGE"
