"""The attention operators write nothing past their buffers: 4 KB of 0xA5 after (and before) every output,
the workspace and the cache's pages stay as they were."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
GUARD = 4096


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


class Guarded:
    """Tensors cut from buffers with guards on both sides."""

    def __init__(self):
        self.all = []

    def make(self, shape, dtype, fill=0):
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        buf = torch.full((GUARD + n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        buf[GUARD:GUARD + n] = fill
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + n:] == 0xA5).all()


@pytest.mark.parametrize("heads,hk,dim,dtype,page", [(28, 4, 128, BF, 16), (40, 8, 128, F8, 7), (32, 8, 64, BF, 24),
                                                     (45, 3, 64, F8, 1), (17, 1, 128, BF, 128)])
def test_append_and_decode(q_, heads, hk, dim, dtype, page):
    lens = [1, 300, 0, 77, 2049]
    g, n = Guarded(), len(lens)
    width = -(-max(lens) // page)
    used = [-(-m // page) for m in lens]
    num = sum(used)
    k, v = (g.make((num, hk, page, dim), dtype) for _ in range(2))
    table = torch.zeros((n, width), dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = torch.arange(at, at + u)
        at += u
    cache = q_.kv_cache(k, v, table.cuda())
    tokens = sum(lens)
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
    seq = torch.repeat_interleave(torch.arange(n, dtype=torch.int32), torch.tensor(lens)).cuda()
    rnd = lambda *s: torch.randn(s, device="cuda").to(BF)
    q, kk, vv = rnd(tokens, heads, dim), rnd(tokens, hk, dim), rnd(tokens, hk, dim)
    qo, ko = g.make((tokens, heads, dim), BF), g.make((tokens, hk, dim), BF)
    ws = g.make((q_.qerl_rope_append_workspace_size(),), torch.uint8)
    freq = torch.linspace(1, 0.001, dim // 2, dtype=torch.float64, device="cuda")
    q_.check(q_.qerl_rope_append(cache, q, kk, vv, pos, freq, qo, ko, ws, seq_ids=seq))
    assert q_.qerl_read_status(ws) == 0
    g.check()
    out, lse = g.make((n, heads, dim), BF), g.make((n, heads), torch.float32)
    dws = g.make((q_.qerl_decode_attention_workspace_size(n, heads, hk, dim),), torch.uint8)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_decode_attention(cache, rnd(n, heads, dim), lengths, 0.1, out, lse, dws))
    assert q_.qerl_read_status(dws) == 0
    g.check()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("heads,hk,dim", [(28, 4, 128), (9, 3, 64)])
@pytest.mark.parametrize("lens", [[1], [130], [700, 3, 0, 257]])
def test_prompt(q_, heads, hk, dim, lens):
    g, t = Guarded(), sum(lens)
    rnd = lambda *s: torch.randn(s, device="cuda").to(BF)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    out, lse = g.make((t, heads, dim), BF, 0xFF), g.make((t, heads), torch.float32, 0xFF)
    ws = g.make((q_.qerl_prompt_attention_workspace_size(t, heads, hk, dim, len(lens)),), torch.uint8)
    q_.check(q_.qerl_prompt_attention(rnd(t, heads, dim), rnd(t, hk, dim), rnd(t, hk, dim), cu, 0.1, out, lse, ws))
    assert q_.qerl_read_status(ws) == 0
    g.check()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()  # every row written
