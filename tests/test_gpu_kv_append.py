"""Rotation of q and k with the append to the paged cache, on the GPU, against the 64-bit form."""
import pytest
import torch

from attention_reference import assert_within, rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _rows(tokens, heads, dim, g, pad=0):
    """bf16 rows of heads, with `pad` elements (NaN) between rows."""
    full = torch.full((tokens, heads * dim + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    full[:, :heads * dim] = torch.randn((tokens, heads * dim), generator=g, device="cuda").to(torch.bfloat16)
    return full[:, :heads * dim].unflatten(1, (heads, dim))


def _freq(half, base=1e4):
    return (base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).cuda()


def _pages(n, hk, page, dim, dtype):
    x = torch.zeros((n, hk, page, dim), dtype=torch.bfloat16, device="cuda")
    return (x + 7).to(dtype)


CASES = [  # heads, kv_heads, dim, rot, page, dtype, pad
    (28, 4, 128, 128, 16, torch.bfloat16, 0),
    (16, 2, 128, 64, 24, torch.float8_e4m3fn, 8),
    (40, 8, 128, 128, 64, torch.float8_e4m3fn, 0),
    (8, 8, 64, 64, 1, torch.bfloat16, 16),
    (45, 3, 64, 16, 7, torch.float8_e4m3fn, 0),
    (3, 1, 64, 0, 128, torch.bfloat16, 0),
    (64, 16, 128, 96, 8, torch.bfloat16, 0),
]


@pytest.mark.parametrize("heads,hk,dim,rot,page,dtype,pad", CASES)
@pytest.mark.parametrize("tokens", [1, 2, 37, 2000])
def test_rotation_and_pages(q_, heads, hk, dim, rot, page, dtype, pad, tokens):
    g = torch.Generator(device="cuda").manual_seed(tokens + heads)
    q, k, v = _rows(tokens, heads, dim, g, pad), _rows(tokens, hk, dim, g, pad), _rows(tokens, hk, dim, g, pad)
    freq = _freq(rot // 2)
    # three sequences, interleaved; positions distinct within each; far ones in the last
    seq = (torch.arange(tokens) % 3).to(torch.int32)
    pos = (torch.arange(tokens) // 3).to(torch.int32)
    pos[seq == 2] += 50000
    pos[4::11] = -1  # padding
    need = [int(pos[seq == s].max()) // page + 1 if (seq == s).any() else 1 for s in range(3)]
    width = max(need)
    touched = sorted({(int(s), int(p) // page) for s, p in zip(seq, pos) if p >= 0})
    num_pages = len(touched) + 2
    table = torch.full((3, width + 3), -5, dtype=torch.int32)  # a padded row stride; the rest is never read
    order = torch.randperm(num_pages, generator=torch.Generator().manual_seed(1)).tolist()
    for i, (s, j) in enumerate(touched):
        table[s, j] = order[i]
    kp, vp = _pages(num_pages, hk, page, dim, dtype), _pages(num_pages, hk, page, dim, dtype)
    e4m3 = dtype != torch.bfloat16
    ks = torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.004 if e4m3 else None
    vs = torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.004 if e4m3 else None
    cache = q_.kv_cache(kp, vp, table.cuda()[:, :width], ks, vs)
    q_out = torch.full((tokens, heads, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((tokens, hk, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    q_.check(q_.qerl_rope_append(cache, q, k, v, pos.cuda(), freq, q_out, k_out, ws, seq_ids=seq.cuda()))
    assert q_.qerl_read_status(ws) == 0

    live = pos >= 0
    lc = live.cuda()
    for name, x, got in (("q", q, q_out), ("k", k, k_out)):
        want, near = rotate64(x[lc], pos[live].cuda(), freq)
        assert_within(got[lc], want, 2.0 ** -8 * want.abs() + near, name)
        assert (got[~lc] == 3.0).all()
    wants = {"k": rotate64(k[lc], pos[live].cuda(), freq), "v": (v[lc].double(), torch.zeros(1, device="cuda"))}
    for name, pages, sc in (("k", kp, ks), ("v", vp, vs)):
        page_of = table[seq[live].long(), (pos[live] // page).long()].long().cuda()
        row = (pos[live] % page).long().cuda()
        got = pages.view(torch.uint8 if e4m3 else torch.bfloat16)[page_of, :, row].view(dtype).float()
        want, near = wants[name]
        if e4m3:
            s = sc.double()[:, None]
            want, near = (want / s).clamp(-448, 448), near / s
            tol = (2.0 ** -4 + 2.0 ** -20) * want.abs() + 2.0 ** -10 + near
        else:
            tol = 2.0 ** -8 * want.abs() + near
        assert_within(got, want, tol, name + " pages")
        # nothing else of the cache changed
        rest = pages.view(torch.uint8 if e4m3 else torch.bfloat16).clone()
        rest[page_of, :, row] = _pages(1, 1, 1, 1, dtype).view(rest.dtype)[0, 0, 0, 0]
        assert torch.equal(rest, _pages(*pages.shape, dtype).view(rest.dtype))


def test_in_place_and_rotation_only(q_):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = _rows(50, 28, 128, g), _rows(50, 4, 128, g)
    pos = torch.randint(0, 2 ** 31 - 1, (50,), generator=g, device="cuda").to(torch.int32)
    freq = _freq(64, 1e6)
    q0, k0 = q.clone(), k.clone()
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    q_.check(q_.qerl_rope_append(None, q, k, None, pos, freq, q, k, ws))
    assert q_.qerl_read_status(ws) == 0
    for x, got in ((q0, q), (k0, k)):
        # the 64-bit angle of a position near 2^31 is itself off by 2^31 2^-53; counted with the fp32 bound
        want, near = rotate64(x, pos, freq)
        assert_within(got, want, 2.0 ** -8 * want.abs() + 2 * near)
    # k alone
    k2 = torch.empty_like(k0)
    q_.check(q_.qerl_rope_append(None, None, k0, None, pos, freq, None, k2, ws))
    assert torch.equal(k2, k)


def test_nan_and_saturation_in_an_8_bit_cache(q_):
    k = torch.full((1, 1, 64), 1e30, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 5], k[0, 0, 6] = float("nan"), -float("inf")
    kp, vp = (torch.zeros((1, 1, 1, 64), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    cache = q_.kv_cache(kp, vp, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    q_.check(q_.qerl_rope_append(cache, None, k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), _freq(0), None,
                                 None, ws))
    assert q_.qerl_read_status(ws) == 0
    for pages in (kp, vp):
        x = pages.float().flatten()
        assert torch.isnan(x[5]) and x[6] == -448
        assert (x[[i for i in range(64) if i not in (5, 6)]] == 448).all()


def test_out_of_range_is_recorded_and_not_written(q_):
    g = torch.Generator(device="cuda").manual_seed(6)
    tokens, hk, dim, page = 6, 2, 64, 4
    k = _rows(tokens, hk, dim, g)
    kp, vp = _pages(3, hk, page, dim, torch.bfloat16), _pages(3, hk, page, dim, torch.bfloat16)
    table = torch.tensor([[0, 1], [-1, 3]], dtype=torch.int32, device="cuda")
    cache = q_.kv_cache(kp, vp, table)
    seq = torch.tensor([0, 1, 1, 2, -1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 0, 4, 0, 0, 8], dtype=torch.int32, device="cuda")
    k_out = torch.empty_like(k)
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    q_.check(q_.qerl_rope_append(cache, None, k, k, pos, _freq(32), None, k_out, ws, seq_ids=seq))
    assert q_.STATUS_NAMES[q_.qerl_read_status(ws)] == "QERL_ERR_RANGE"
    assert q_.qerl_read_status(ws) == 0
    want, near = rotate64(k, pos, _freq(32))  # the rotation itself is done
    assert_within(k_out, want, 2.0 ** -8 * want.abs() + near)
    assert torch.equal(kp[1, :, 1], k_out[0])
    kp[1, :, 1] = 7
    assert (kp == 7).all()  # only the good token was appended


def test_empty_and_stream(q_):
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    q_.check(q_.qerl_rope_append(None, None, e, None, torch.empty(0, dtype=torch.int32, device="cuda"), _freq(32), None,
                                 e, ws))
    g = torch.Generator(device="cuda").manual_seed(7)
    k = _rows(33, 4, 64, g)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(k), torch.empty_like(k)
    q_.check(q_.qerl_rope_append(None, None, k, None, pos, _freq(32), None, a, ws))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q_.check(q_.qerl_rope_append(None, None, k, None, pos, _freq(32), None, b, ws, stream=s))
    s.synchronize()
    assert torch.equal(a, b)
