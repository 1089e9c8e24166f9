"""The rollout example: tokens generated one at a time over the paged cache give what one causal pass
over the whole sequences gives.

Bounds (relative norm of the block's output).  Both passes round q, k, v, the attention's output and
the o linear's to bf16 (half a step 2^-8 each); the values enter both the same way, so what differs is
the rounding of the softmax weights (2^-8 at most in the causal pass), the linears' accumulation
order, which moves a bf16 rounding by a step now and then, and each output's own rounding: below
4 half steps, 2^-6.  An E4M3 cache rounds k and v by up to 2^-4: each of the two moves the attention's
output by at most that, relative to sums of magnitudes that random signs make a few times larger than
the output, and the residual, which is larger than the branch, is exact: 2^-2.
"""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("dtype,bound", [(torch.bfloat16, 2.0 ** -6), (torch.float8_e4m3fn, 2.0 ** -2)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (14, 2, 64)])
def test_steps_match_one_causal_pass(dtype, bound, heads, kv_heads, dim):
    from rollout_block import rollout
    got, want, us = rollout(heads, kv_heads, dim, cache_dtype=dtype)
    assert len(got) == 6 and us > 0
    for t, (a, b) in enumerate(zip(got, want)):
        assert torch.isfinite(a.float()).all()
        far = ((a.float() - b.float()).norm() / b.float().norm()).item()
        assert far <= bound, f"step {t}: {far:.3e}"
