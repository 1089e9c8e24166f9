"""The window, tree and page operators write nothing past their buffers: 4 KB of 0xA5 after (and before) every
output, the workspace, the table and the cache's pages stay as they were."""
import pytest
import torch

from test_gpu_attention_guards import Guarded

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rnd(*shape):
    return torch.randn(shape, device="cuda").to(BF)


def _cache(q_, g, lens, hk, dim, dtype, page, spare=0, rows=0):
    used = [-(-m // page) for m in lens]
    k, v = (g.make((sum(used) + spare, hk, page, dim), dtype) for _ in range(2))
    table = g.make((len(lens) + rows, max(used)), torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = torch.arange(at, at + u)
        at += u
    return q_.kv_cache(k, v, table), at


SHAPES = [(28, 4, 128, BF, 16), (40, 8, 128, F8, 7), (32, 8, 64, BF, 24), (45, 3, 64, F8, 1), (17, 1, 128, BF, 128)]


@pytest.mark.parametrize("heads,hk,dim,dtype,page", SHAPES)
def test_window_decode_and_tree(q_, heads, hk, dim, dtype, page):
    lens, counts = [1, 300, 0, 77, 2049], [1, 40, 7, 0, 130]
    g, n, t = Guarded(), len(lens), sum(counts)
    cache, _ = _cache(q_, g, lens, hk, dim, dtype, page)
    out, lse = g.make((n, heads, dim), BF, 0xFF), g.make((n, heads), torch.float32, 0xFF)
    ws = g.make((q_.qerl_decode_attention_workspace_size(n, heads, hk, dim),), torch.uint8)
    q_.check(q_.qerl_window_decode_attention(cache, _rnd(n, heads, dim), _i32(lens), 100, 5, 0.1, out, lse, ws))
    assert q_.qerl_read_status(ws) == 0
    g.check()
    assert torch.isfinite(out).all()
    out, lse = g.make((t, heads, dim), BF, 0xFF), g.make((t, heads), torch.float32, 0xFF)
    ws = g.make((q_.qerl_tree_attention_workspace_size(t, heads, hk, dim, n),), torch.uint8)
    cu = _i32([0] + torch.tensor(counts).cumsum(0).tolist())
    for mask in (None, torch.full((t, 3), -1, dtype=torch.int64, device="cuda")):
        q_.check(q_.qerl_tree_attention(cache, _rnd(t, heads, dim), _rnd(t, hk, dim), _rnd(t, hk, dim), cu, _i32(lens), mask,
                                        0.1, out, lse, ws))
        assert q_.qerl_read_status(ws) == 0
        g.check()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()  # every row written


@pytest.mark.parametrize("heads,hk,dim", [(28, 4, 128), (9, 3, 64)])
@pytest.mark.parametrize("lens", [[1], [130], [700, 3, 0, 257]])
def test_window_prompt(q_, heads, hk, dim, lens):
    g, t = Guarded(), sum(lens)
    cu = _i32([0] + torch.tensor(lens).cumsum(0).tolist())
    out, lse = g.make((t, heads, dim), BF, 0xFF), g.make((t, heads), torch.float32, 0xFF)
    ws = g.make((q_.qerl_prompt_attention_workspace_size(t, heads, hk, dim, len(lens)),), torch.uint8)
    q_.check(q_.qerl_window_prompt_attention(_rnd(t, heads, dim), _rnd(t, hk, dim), _rnd(t, hk, dim), cu, 60, 3, 0.1, out,
                                             lse, ws))
    assert q_.qerl_read_status(ws) == 0
    g.check()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()  # every row written


@pytest.mark.parametrize("heads,hk,dim,dtype,page", SHAPES)
def test_fork_and_compact(q_, heads, hk, dim, dtype, page):
    lens = [1, 300, 77, 2049]
    g, n = Guarded(), len(lens)
    cache, used = _cache(q_, g, lens, hk, dim, dtype, page, spare=n + 3, rows=n)
    ws = g.make((q_.qerl_kv_fork_workspace_size(),), torch.uint8)
    q_.check(q_.qerl_kv_fork(cache, _i32(list(range(n))), _i32(list(range(n, 2 * n))), _i32(lens),
                             _i32([used + 3 + i for i in range(n)]), ws))
    assert q_.qerl_read_status(ws) == 0
    g.check()
    new, live = g.make((2 * n, cache.max_pages), torch.int32), g.make((1,), torch.int32)
    ws = g.make((q_.qerl_kv_compact_workspace_size(cache.num_pages),), torch.uint8)
    q_.check(q_.qerl_kv_compact(cache, _i32([0, 300, 0, 0, 1, 0, 77, 2049]), new, live, ws))
    assert q_.qerl_read_status(ws) == 0
    g.check()
