"""Attention of one new token over an E4M3 cache where its 16-bit operands could lose what matters, and
the joins of segments cut over many CTAs for every head layout.

Bounds: those of attention_reference, with the loss of tiny weights counted as the kernel has it: a weight
is held to half a step of fp16, 2^-11 relative or 2^-25 where its steps are even, of weights that are 2^7
at the running reference, so 2^-32 of the largest weight."""
import math

import pytest
import torch

from attention_reference import assert_within, attend64

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _paged(rows, page, seed):
    """[hk, n, dim] of one sequence -> (pages in a shuffled order, table)."""
    hk, n, dim = rows[0].shape
    used = -(-n // page)
    order = torch.randperm(used, generator=torch.Generator().manual_seed(seed)).cuda()
    out = []
    for x in rows:
        raw = x.view(torch.uint8) if x.dtype == F8 else x
        full = torch.zeros((hk, used * page, dim), dtype=raw.dtype, device="cuda")
        full[:, :n] = raw
        pages = torch.empty((used, hk, page, dim), dtype=raw.dtype, device="cuda")
        pages[order] = full.view(hk, used, page, dim).transpose(0, 1)
        out.append(pages.view(x.dtype))
    return out, order.to(torch.int32)[None]


def _run(q_, cache, q, lens, scale):
    n, h, d = q.shape
    out, lse = torch.full_like(q, float("nan")), torch.full((n, h), float("nan"), device="cuda")
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(n, h, cache.num_kv_heads, d))
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_decode_attention(cache, q, lengths, scale, out, lse, ws))
    assert q_.qerl_read_status(ws) == 0
    return out, lse, ws


HEADS = [(4, 1, 64), (12, 1, 64), (4, 1, 128), (12, 1, 128)]


@pytest.mark.parametrize("heads,hk,dim", HEADS)
@pytest.mark.parametrize("bits", [20.0, 24.5, 26.5, 28.0])
def test_many_tiny_weights_are_not_lost(q_, heads, hk, dim, bits):
    """Every 16th key has the largest weight and a value of 0, the others 2^-bits of it and a value of 1:
    the output is 15 * 2^-bits, and nothing else."""
    n = 4096
    k, v = torch.zeros((1, n, dim), device="cuda"), torch.ones((1, n, dim), device="cuda")
    k[:, :, 0] = -16.0
    k[:, ::16] = 0.0
    v[:, ::16] = 0.0
    k, v = k.to(F8), v.to(F8)
    (kp, vp), table = _paged((k, v), 16, 0)
    q = torch.zeros((1, heads, dim), dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    scale = bits * math.log(2.0) / 16.0
    out, lse, _ = _run(q_, q_.kv_cache(kp, vp, table), q, [n], scale)
    want, l, _, tl = attend64(q[0], k[0], v[0], scale, "fp16")
    # scores to 2^-20 (1 + 16 scale) each; the weights as above, 16 of them for each largest one
    d = 2.0 ** -20 * (1.0 + 16.0 * scale)
    tol = (2.0 ** -8 + 2.0 * (2.0 * d + 2.0 ** -11)) * want + 16 * 2.0 ** -32
    assert (want > 2 * tol).all()
    assert_within(out[0], want, tol, "output")
    assert_within(lse[0], l, tl, "lse")


@pytest.mark.parametrize("heads,hk,dim", HEADS)
@pytest.mark.parametrize("below", [10, 16, 20, 22])
def test_query_elements_far_below_the_largest(q_, heads, hk, dim, below):
    """The largest query element meets keys that are 0 there; the scores come from elements 2^-below of it."""
    n = 500
    g = torch.Generator(device="cuda").manual_seed(below + dim)
    k = torch.randn((1, n, dim), generator=g, device="cuda")
    k[:, :, 0] = 0.0
    v = torch.randn((1, n, dim), generator=g, device="cuda")
    k, v = k.to(F8), v.to(F8)
    (kp, vp), table = _paged((k, v), 16, 1)
    q = (torch.randn((1, heads, dim), generator=g, device="cuda") * 2.0 ** -below).to(BF)
    q[:, :, 0] = 1.0
    scale = 2.0 ** below / math.sqrt(dim)
    out, lse, _ = _run(q_, q_.kv_cache(kp, vp, table), q, [n], scale)
    want, l, tol, tl = attend64(q[0], k[0], v[0], scale, "fp16")
    assert_within(out[0], want, tol, "output")
    assert_within(lse[0], l, tl, "lse")


@pytest.mark.parametrize("heads,hk,dim", HEADS)
def test_an_infinite_query_element_beside_large_ones(q_, heads, hk, dim):
    """Every score is -inf: an empty row, though the head's finite elements are large."""
    n = 200
    g = torch.Generator(device="cuda").manual_seed(dim)
    k, v = torch.randn((1, n, dim), generator=g, device="cuda"), torch.randn((1, n, dim), generator=g, device="cuda")
    k[:, :, 3] = 1.0
    (kp, vp), table = _paged((k.to(F8), v.to(F8)), 16, 2)
    q = torch.zeros((1, heads, dim), dtype=BF, device="cuda")
    q[:, :, 3], q[:, :, 5], q[:, :, 6] = -math.inf, 1e38, 1e30
    out, lse, _ = _run(q_, q_.kv_cache(kp, vp, table), q, [n], 1e-3)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("heads,hk,dim", [(8, 2, 64), (45, 3, 64), (12, 1, 128), (40, 1, 128), (40, 8, 128), (17, 1, 64)])
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("n", [30011, 6001])
def test_segments_over_many_ctas(q_, heads, hk, dim, dtype, n):
    """One sequence whose (sequence, head) segments are cut over up to hundreds of CTAs and joined in one or
    two levels; the same bit for bit when the workspace is used again."""
    g = torch.Generator(device="cuda").manual_seed(n + heads)
    rows = [torch.randn((hk, n, dim), generator=g, device="cuda").to(dtype) for _ in range(2)]
    (kp, vp), table = _paged(rows, 32, 3)
    q = (torch.randn((1, heads, dim), generator=g, device="cuda") * 1.5).to(BF)
    scale = 1 / math.sqrt(dim)
    cache = q_.kv_cache(kp, vp, table)
    out, lse, ws = _run(q_, cache, q, [n], scale)
    group = heads // hk
    for j in range(hk):
        mine = slice(j * group, (j + 1) * group)
        o, l, to, tl = attend64(q[0, mine], rows[0][j], rows[1][j], scale, "split" if dtype == BF else "fp16")
        assert_within(out[0, mine], o, to, f"head {j}")
        assert_within(lse[0, mine], l, tl, f"lse of head {j}")
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    for _ in range(3):
        q_.check(q_.qerl_decode_attention(cache, q, lengths, scale, again, lse2, ws))
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert q_.qerl_read_status(ws) == 0
