"""Causal attention of packed whole prompts, on the GPU, against the 64-bit form."""
import math

import pytest
import torch

from attention_reference import assert_within, causal64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _rows(tokens, heads, dim, g, std=1.0, pad=0):
    """bf16 rows of heads with `pad` NaN elements between rows."""
    full = torch.full((tokens, heads * dim + pad), float("nan"), dtype=BF, device="cuda")
    full[:, :heads * dim] = (torch.randn((tokens, heads * dim), generator=g, device="cuda") * std).to(BF)
    return full[:, :heads * dim].unflatten(1, (heads, dim))


def _cu(lens, lead=0):
    cu = [lead]
    for m in lens:
        cu.append(cu[-1] + m)
    return torch.tensor(cu, dtype=torch.int32, device="cuda"), cu


def _run(q_, q, k, v, cu, scale, stream=None, pad=0):
    t, h, d = q.shape
    out = torch.full((t, h * d + pad), 5.0, dtype=BF, device="cuda")[:, :h * d].unflatten(1, (h, d))
    lse = torch.full((t, h), 5.0, device="cuda")
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(t, h, k.shape[1], d, cu.numel() - 1))
    if stream is not None:
        torch.cuda.synchronize()
    q_.check(q_.qerl_prompt_attention(q, k, v, cu, scale, out, lse, ws, stream=stream))
    assert q_.qerl_read_status(ws, stream=stream) == 0
    return out, lse


def _check(q, k, v, cu, scale, out, lse):
    group = q.shape[1] // k.shape[1]
    for i in range(len(cu) - 1):
        rows = slice(cu[i], cu[i + 1])
        if cu[i] == cu[i + 1]:
            continue
        for h in range(q.shape[1]):
            o, l, to, tl = causal64(q[rows, h], k[rows, h // group], v[rows, h // group], scale, "bf16")
            assert_within(out[rows, h], o, to, f"sequence {i} head {h}")
            assert_within(lse[rows, h], l, tl, f"lse of sequence {i} head {h}")


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255], [256], [257], [640], [1000], [2111],
                                  [1, 0, 300, 77, 128, 256, 0, 513, 5, 1]])
@pytest.mark.parametrize("heads,hk,dim", [(28, 4, 128), (5, 1, 64), (4, 4, 128), (9, 3, 64)])
def test_lengths_and_groups(q_, lens, heads, hk, dim):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + heads)
    t = sum(lens)
    q, k, v = _rows(t, heads, dim, g, 1.5), _rows(t, hk, dim, g), _rows(t, hk, dim, g)
    cu, cu_list = _cu(lens)
    scale = 1 / math.sqrt(dim)
    out, lse = _run(q_, q, k, v, cu, scale)
    _check(q, k, v, cu_list, scale, out, lse)


def test_strides_gaps_and_determinism(q_):
    """Padded row strides; rows before the first and after the last sequence are not touched."""
    g = torch.Generator(device="cuda").manual_seed(3)
    heads, hk, dim, lens, lead, tail = 8, 2, 128, [300, 41, 129], 7, 30
    t = lead + sum(lens) + tail
    q, k, v = _rows(t, heads, dim, g, 1.5, 8), _rows(t, hk, dim, g, 1.0, 16), _rows(t, hk, dim, g, 1.0, 24)
    cu, cu_list = _cu(lens, lead)
    out, lse = _run(q_, q, k, v, cu, 0.09, pad=40)
    _check(q, k, v, cu_list, 0.09, out, lse)
    for x in (out, lse):
        assert (x[:lead] == 5).all() and (x[-tail:] == 5).all()
    again, lse2 = _run(q_, q, k, v, cu, 0.09, stream=torch.cuda.Stream())
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.2, 1.0), (2.0, 3.0), (0.5, 8.0)])
def test_flat_negative_and_peaked_scores(q_, scale, std):
    g = torch.Generator(device="cuda").manual_seed(4)
    heads, hk, dim, lens = 4, 2, 128, [700, 90]
    t = sum(lens)
    q, k, v = _rows(t, heads, dim, g, std), _rows(t, hk, dim, g), _rows(t, hk, dim, g)
    cu, cu_list = _cu(lens)
    out, lse = _run(q_, q, k, v, cu, scale)
    _check(q, k, v, cu_list, scale, out, lse)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_growing_scores(q_, sign):
    """Scores that rise along the keys: the reference moves in every tile and O is rescaled."""
    n, dim = 1500, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.zeros((n, 2, dim), dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros((n, 1, dim), dtype=BF, device="cuda")
    k[:, 0, 0] = (torch.arange(n, device="cuda") * 0.25).to(BF)
    v = _rows(n, 1, dim, g)
    cu, cu_list = _cu([n])
    out, lse = _run(q_, q, k, v, cu, sign)
    _check(q, k, v, cu_list, sign, out, lse)


def test_non_finite_rows_reach_only_later_rows(q_):
    """NaN and infinities in k and v: rows before them, other sequences and other heads' outputs are what
    they are without them; rows from them on are non-finite."""
    g = torch.Generator(device="cuda").manual_seed(6)
    heads, hk, dim, lens = 4, 2, 128, [600, 130, 20]
    t = sum(lens)
    cu, cu_list = _cu(lens)
    q, k, v = _rows(t, heads, dim, g, 1.5), _rows(t, hk, dim, g), _rows(t, hk, dim, g)
    for row, what, name in [(600 + 5, float("nan"), "v"), (40, float("nan"), "v"), (129, float("inf"), "v"),
                            (300, -float("inf"), "v"), (511, float("nan"), "k"), (599, float("inf"), "v"),
                            (600 + 129, float("nan"), "k"), (730, float("nan"), "v")]:
        k2, v2 = k.clone(), v.clone()
        (v2 if name == "v" else k2)[row, 1, 3] = what
        out, lse = _run(q_, q, k2, v2, cu, 0.09)
        kz, vz = k2.clone(), v2.clone()
        (vz if name == "v" else kz)[row, 1, 3] = 0  # the rows before it do not see what it holds
        end = [c for c in cu_list if c > row][0]
        hurt = torch.zeros((t, heads), dtype=torch.bool, device="cuda")
        hurt[row:end, 2:] = True
        hurt_out = hurt[:, :, None].expand(t, heads, dim).clone()
        if name == "v":  # only that element of the outputs; the sums do not see v
            hurt_out[:] = False
            hurt_out[row:end, 2:, 3] = True
            hurt[:] = False
        assert not torch.isfinite(out[hurt_out]).any()
        assert torch.isfinite(out[~hurt_out]).all()
        assert not torch.isfinite(lse[hurt]).any() and torch.isfinite(lse[~hurt]).all()
        for i in range(len(lens)):
            rows = slice(cu_list[i], cu_list[i + 1])
            for h in range(heads):
                o, l, to, tl = causal64(q[rows, h], kz[rows, h // 2], vz[rows, h // 2], 0.09, "bf16")
                good = ~hurt_out[rows, h]
                assert_within(out[rows, h][good], o[good], to[good], f"{name} {what} at {row}")
                good = ~hurt[rows, h]
                assert_within(lse[rows, h][good], l[good], tl[good], f"lse, {name} {what} at {row}")


def test_many_short_prompts(q_):
    """More sequences than a warp has lanes, in an order that is not sorted."""
    lens = [(i * 37) % 300 for i in range(150)]
    g = torch.Generator(device="cuda").manual_seed(7)
    t = sum(lens)
    q, k, v = _rows(t, 2, 64, g, 1.5), _rows(t, 1, 64, g), _rows(t, 1, 64, g)
    cu, cu_list = _cu(lens)
    out, lse = _run(q_, q, k, v, cu, 0.125)
    _check(q, k, v, cu_list, 0.125, out, lse)


def test_many_empty_and_equal_prompts(q_):
    """Hundreds of sequences, most of them empty, some a block, some two: every block is found once."""
    lens = [0] * 400
    for i in range(0, 400, 3):
        lens[i] = 1 + (i * 11) % 40
    lens[200], lens[7] = 300, 513
    g = torch.Generator(device="cuda").manual_seed(10)
    t = sum(lens)
    q, k, v = _rows(t, 4, 64, g, 1.5), _rows(t, 2, 64, g), _rows(t, 2, 64, g)
    cu, cu_list = _cu(lens)
    out, lse = _run(q_, q, k, v, cu, 0.125)
    _check(q, k, v, cu_list, 0.125, out, lse)


def test_no_lse(q_):
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = _rows(300, 4, 128, g), _rows(300, 2, 128, g), _rows(300, 2, 128, g)
    cu, _ = _cu([300])
    out, _ = _run(q_, q, k, v, cu, 0.09)
    again = torch.empty_like(out)
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(300, 4, 2, 128, 1))
    q_.check(q_.qerl_prompt_attention(q, k, v, cu, 0.09, again, None, ws))
    assert q_.qerl_read_status(ws) == 0 and torch.equal(out, again)


def test_bad_offsets_are_recorded(q_):
    g = torch.Generator(device="cuda").manual_seed(8)
    t = 100
    q, k, v = _rows(t, 2, 64, g), _rows(t, 1, 64, g), _rows(t, 1, 64, g)
    out, lse = torch.zeros_like(q), torch.zeros((t, 2), device="cuda")
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(t, 2, 1, 64, 2))
    for cu in ([0, 101, 101], [-1, 50, 100], [0, 60, 40], [0, 2 ** 31 - 1, 2 ** 31 - 1]):
        q_.check(q_.qerl_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 0.125, out, lse,
                                          ws))
        assert q_.STATUS_NAMES[q_.qerl_read_status(ws)] == "QERL_ERR_RANGE"
        assert q_.qerl_read_status(ws) == 0


def test_graph(q_):
    g = torch.Generator(device="cuda").manual_seed(9)
    lens = [333, 12]
    t = sum(lens)
    q, k, v = _rows(t, 4, 128, g), _rows(t, 2, 128, g), _rows(t, 2, 128, g)
    cu, cu_list = _cu(lens)
    a, la = _run(q_, q, k, v, cu, 0.09)
    out, lse = torch.zeros_like(a), torch.zeros_like(la)
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(t, 4, 2, 128, 2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q_.check(q_.qerl_prompt_attention(q, k, v, cu, 0.09, out, lse, ws))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
