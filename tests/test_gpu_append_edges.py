"""The append at its edges: a cache without pages, scales whose reciprocal leaves fp32's range, no queries, and
the 8-bit values bit for bit."""
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


# Scales of every size; values whose quotients are 0, E4M3 values, or past its largest, so nothing is rounded.
@pytest.mark.parametrize("exponent", [-149, -140, -130, -127, -126, -120, -64, -9, 0, 30, 64, 100, 126, 127])
def test_scales_whose_reciprocal_is_out_of_range(q_, exponent):
    dim = 128
    quotients = [0.0] + [(1.0 + (i % 8) / 8.0) * 2.0 ** (i // 8 - 6) * (-1) ** i for i in range(1, 120)]
    quotients += [2.0 ** e for e in (10, 16, 17, 20, 30, 60, 100, -11)]
    x = torch.tensor(quotients, dtype=torch.float64) * 2.0 ** exponent
    held = (x.abs() < 2.0 ** 128) & (x.to(BF).double() == x)  # by bf16, subnormals included
    x = torch.where(held, x, 0.0)
    want = (x / 2.0 ** exponent).clamp(-448, 448).float()
    want[want.abs() == 2.0 ** -11] = 0.0  # half of E4M3's smallest step is 2^-10
    k = x.to(BF).view(1, 1, dim).cuda()
    assert (want == 0).any() and (want != 0).sum() >= (3 if exponent < -135 else 20)
    kp, vp = (torch.full((1, 1, 1, dim), 0x7F, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    scale = torch.tensor([2.0 ** exponent], dtype=torch.float64).float().cuda()
    assert scale.item() == 2.0 ** exponent
    cache = q_.kv_cache(kp, vp, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), scale, scale)
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    q_.check(q_.qerl_rope_append(cache, None, k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), _no_freq(), None,
                                 None, ws))
    assert q_.qerl_read_status(ws) == 0
    for pages in (kp, vp):
        assert torch.equal(pages.float().flatten().cpu(), want)


def test_rope_append_without_queries(q_):
    """The Python call takes no q where the entry point does."""
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn((5, 2, 64), generator=g, device="cuda").to(BF)
    pages = [torch.zeros((2, 2, 4, 64), dtype=BF, device="cuda") for _ in range(2)]
    cache = q_.kv_cache(*pages, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    freq = torch.linspace(1, 0.01, 32, dtype=torch.float64, device="cuda")
    none, k_out = q_.rope_append(cache, None, k, k, pos, freq, seq_ids=torch.zeros_like(pos))
    assert none is None
    q_out, k_too = q_.rope_append(None, k, k, None, pos, freq)
    assert torch.equal(k_out, k_too) and torch.equal(q_out, k_too)
    assert torch.equal(pages[0][1].transpose(0, 1), k_out[:4]) and torch.equal(pages[1][0, :, 0], k[4])


def test_rope_append_gives_zeros_for_padding(q_):
    """Not what the memory held before."""
    k = torch.ones((4000, 8, 128), dtype=BF, device="cuda")
    pos = torch.full((4000,), -1, dtype=torch.int32, device="cuda")
    pos[7] = 3
    for _ in range(2):
        dirt = torch.full_like(k, float("nan")), torch.full_like(k, float("nan"))
        torch.cuda.synchronize()
        del dirt  # the allocator hands the same memory out again
        q_out, k_out = q_.rope_append(None, k, k, None, pos, _no_freq())
        for x in (q_out, k_out):
            assert (x[7] == 1).all()
            x[7] = 0
            assert (x == 0).all()


@pytest.mark.parametrize("hk,dim", [(1, 64), (8, 128), (3, 64)])
def test_8_bit_values_bit_for_bit(q_, hk, dim):
    """v is not rotated: its bytes are those of value * (1 / scale), both steps in fp32, rounded to nearest
    even and clamped to +-448."""
    tokens, page = 700, 16
    g = torch.Generator(device="cuda").manual_seed(hk)
    v = (torch.randn((tokens, hk, dim), generator=g, device="cuda") *
         2.0 ** torch.randint(-14, 6, (tokens, 1, 1), generator=g, device="cuda")).to(BF)
    v[0] = 0.0
    v[1] = -0.0
    vs = torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.003
    vs[0] = 1.0 / 64  # quotients that are exact, so midpoints between E4M3 values are met
    v[2:200, 0] = (torch.randint(-256, 257, (198, dim), generator=g, device="cuda") / 512.0).to(BF)
    kp, vp = (torch.zeros((-(-tokens // page), hk, page, dim), dtype=torch.uint8, device="cuda").view(F8)
              for _ in range(2))
    table = torch.arange(kp.shape[0], dtype=torch.int32, device="cuda")[None]
    cache = q_.kv_cache(kp, vp, table, vs, vs)
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_rope_append(cache, None, v, v, pos, _no_freq(), None, None, ws, seq_ids=torch.zeros_like(pos)))
    assert q_.qerl_read_status(ws) == 0
    quotient = v.float() * (1.0 / vs)[None, :, None]
    want = quotient.clamp(-448, 448).to(F8).view(torch.uint8)
    assert ((quotient * 2.0 ** 12).frac() == 0).any()
    for pages in (kp, vp):
        got = pages.view(torch.uint8).transpose(1, 2).reshape(-1, hk, dim)[:tokens]
        assert torch.equal(got, want)
