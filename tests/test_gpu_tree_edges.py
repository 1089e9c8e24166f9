"""Attention of drafted tokens where small weights, scales, neighbouring rows or the number of sequences could show.

Bound of an output over an E4M3 cache: that of masked_reference, with the roundings of the weights counted as the
kernel has them and without its factor for the division, as their sum is taken of unrounded ones.  Weights of the
cache's rows are rounded to fp16, 2^-11 relative or 2^-25 where its steps are even, of weights of which the largest
is at least 2^7, so 2^-32 of the largest; those of the new tokens to bf16, 2^-8."""
import math
import random

import pytest
import torch

from attention_reference import assert_within
from masked_reference import masked64
from test_gpu_tree_attention import BF, F8, Case, _i32, q_  # noqa: F401 (q_ is a fixture)

pytestmark = pytest.mark.gpu


def mixed64(q, k, v, scale, keep, rows):
    """masked64 over an E4M3 cache: the first `rows` keys are the cache's, the others the new tokens'."""
    out, lse, _, tol_lse = masked64(q, k, v, scale, keep, "split")
    q, k, v = q.double(), k.double(), v.double()
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    s = torch.where(keep, (q @ k.T) * scale, zero - math.inf)
    p = torch.where(keep, torch.exp(s - torch.where(keep.any(1), lse, zero)[:, None]), zero)
    d = 2.0 ** -20 * (1.0 + abs(scale) * torch.where(keep, q.abs() @ k.abs().T, zero).amax(1))
    mine, new = (p[:, x] @ v[x].abs() for x in (slice(rows), slice(rows, None)))
    tol = 2.0 ** -8 * out.abs() + 4.0 * d[:, None] * (mine + new) + 2.0 ** -11 * mine + 2.0 ** -8 * new
    if rows:
        tol = tol + rows * 2.0 ** -32 * p[:, :rows].amax(1)[:, None] * v[:rows].abs().amax(0)
    return out, lse, tol + 1e-30, tol_lse


# ---- weights over an E4M3 cache ----------------------------------------------


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("count", [1, 140])
@pytest.mark.parametrize("bits", [20.0, 24.5, 26.5, 28.0])
def test_many_tiny_weights_are_not_lost(q_, dim, count, bits):
    """Every 1024th key has the largest weight and a value of 0, the others 2^-bits of it and a value of 1.  The
    sequences are one and the same, so many that CTAs hold whole segments."""
    n, hk, seqs = 16384, 4, 50
    k, v = torch.zeros((hk, n, dim), device="cuda"), torch.ones((hk, n, dim), device="cuda")
    k[:, :, 0] = -16.0
    k[:, ::1024] = 0.0
    v[:, ::1024] = 0.0
    pages = [x.to(F8).view(torch.uint8).view(hk, n // 64, 64, dim).transpose(0, 1).contiguous().view(F8) for x in (k, v)]
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    q = torch.zeros((count * seqs, hk, dim), dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    new = torch.ones((count * seqs, hk, dim), dtype=BF, device="cuda")
    mask = torch.zeros((count * seqs, 3), dtype=torch.int64, device="cuda")  # no new token is seen
    scale = bits * math.log(2.0) / 16.0
    out, lse = q_.tree_attention(q_.kv_cache(*pages, table), q, new, new, _i32([count * s for s in range(seqs + 1)]),
                                 _i32([n] * seqs), mask, scale)
    keep = torch.ones((1, n), dtype=torch.bool, device="cuda")
    o, l, to, tl = mixed64(q[0, :1], k[0], v[0], scale, keep, n)
    assert (o > 2 * to).all()
    assert_within(out, o.expand_as(out), to.expand_as(out), "output")
    assert_within(lse, l.expand_as(lse), tl.expand_as(lse), "lse")
