"""The rollout example's attention branch (output minus residual) in the two passes.

The residual is exact and several times the branch, so a bound on the whole output says little about the
attention.  Bounds on the difference of the branches, as norms:

  the outputs' own roundings   2 * 2^-8 |output|   (half a step each, of residual plus branch)
  bf16 cache                   2^-6 |branch|       (softmax weights, the attention's and the o linear's outputs,
                                                    a step of the linears now and then: 4 half steps)
  E4M3 cache                   2^-3 |branch|       (the above; v off by up to 2^-4 of itself, independently from
                                                    row to row as the rows are, so the weighted sum is off by at
                                                    most that part of its size; k moves the scores, of size 1, by
                                                    less, and the weights with them)

Attention that gave nothing, or another sequence's, would be off by all of the branch."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("dtype,part", [(torch.bfloat16, 2.0 ** -6), (torch.float8_e4m3fn, 2.0 ** -3)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (14, 2, 64)])
def test_branches_match(dtype, part, heads, kv_heads, dim):
    import workloads as wl
    from rollout_block import rollout
    lens, steps, seed = (37, 5, 130, 64), 6, 0
    got, want, _ = rollout(heads, kv_heads, dim, lens, steps, dtype, seed)
    total = [m + steps for m in lens]
    hidden = wl.normal_bf16_device((sum(total), heads * dim), 1.0, seed, 77)
    start = [sum(total[:i]) for i in range(len(lens))]
    for t, (a, b) in enumerate(zip(got, want)):
        residual = torch.stack([hidden[s + m + t] for s, m in zip(start, lens)]).double()
        branch = b.double() - residual
        assert branch.norm() > 2.0 ** -4 * residual.norm()
        far = (a.double() - b.double()).norm()
        bound = part * branch.norm() + 2 * 2.0 ** -8 * b.double().norm()
        assert bound < 0.25 * branch.norm() and far <= bound, f"step {t}: {far:.3e} of {bound:.3e}, {branch.norm():.3e}"
