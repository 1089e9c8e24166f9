"""Attention within a window, with sinks: packed prompts and one new token per sequence, against the 64-bit form."""
import math

import pytest
import torch

from attention_reference import assert_within
from masked_reference import masked64, window_keep

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


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


# ---- packed prompts ---------------------------------------------------------


def _offsets(lens, lead=0):
    cu = [lead]
    for m in lens:
        cu.append(cu[-1] + m)
    return cu


def _prompt(q_, q, k, v, cu, window, sinks, scale, stream=None):
    t, h, d = q.shape
    out, lse = torch.full((t, h, d), 5.0, dtype=BF, device="cuda"), torch.full((t, h), 5.0, device="cuda")
    ws = q_.workspace(q_.qerl_prompt_attention_workspace_size(t, h, k.shape[1], d, len(cu) - 1))
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    q_.check(q_.qerl_window_prompt_attention(q, k, v, cu, window, sinks, scale, out, lse, ws, stream=stream))
    assert q_.qerl_read_status(ws, stream=stream) == 0
    return out, lse


def _check_prompt(q, k, v, cu, window, sinks, scale, out, lse):
    group = q.shape[1] // k.shape[1]
    for i in range(len(cu) - 1):
        rows = slice(cu[i], cu[i + 1])
        if cu[i] == cu[i + 1]:
            continue
        at = torch.arange(cu[i + 1] - cu[i], device="cuda")
        keep = window_keep(at, at, window, sinks)
        for h in range(q.shape[1]):
            o, l, to, tl = masked64(q[rows, h], k[rows, h // group], v[rows, h // group], scale, keep, "bf16")
            assert_within(out[rows, h], o, to, f"sequence {i} head {h}")
            assert_within(lse[rows, h], l, tl, f"lse of sequence {i} head {h}")


LENS = [1, 0, 300, 77, 128, 256, 0, 1101, 5, 1]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (64, 0), (127, 3), (128, 0), (129, 128), (130, 129),
                                          (200, 500), (255, 4), (256, 0), (257, 1), (384, 130), (1000, 4), (1100, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 31 - 1)])
@pytest.mark.parametrize("heads,hk,dim", [(4, 2, 128), (3, 1, 64)])
def test_prompt_windows(q_, window, sinks, heads, hk, dim):
    g = torch.Generator(device="cuda").manual_seed(window % 1000 + sinks % 1000 + heads)
    t = sum(LENS)
    q, k, v = _rows(t, heads, dim, g, 1.5), _rows(t, hk, dim, g), _rows(t, hk, dim, g)
    cu = _offsets(LENS)
    out, lse = _prompt(q_, q, k, v, cu, window, sinks, 1 / math.sqrt(dim))
    _check_prompt(q, k, v, cu, window, sinks, 1 / math.sqrt(dim), out, lse)


def test_prompt_long_with_strides_gaps_and_another_stream(q_):
    g = torch.Generator(device="cuda").manual_seed(3)
    heads, hk, dim, lens, lead, tail = 14, 2, 128, [2500, 41, 1290], 7, 30
    t = lead + sum(lens) + tail
    q, k, v = _rows(t, heads, dim, g, 1.5, 8), _rows(t, hk, dim, g, 1.0, 16), _rows(t, hk, dim, g, 1.0, 24)
    cu = _offsets(lens, lead)
    out, lse = _prompt(q_, q, k, v, cu, 300, 10, -0.09)
    _check_prompt(q, k, v, cu, 300, 10, -0.09, out, lse)
    for x in (out, lse):
        assert (x[:lead] == 5).all() and (x[-tail:] == 5).all()
    again, lse2 = _prompt(q_, q, k, v, cu, 300, 10, -0.09, stream=torch.cuda.Stream())
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [[130, 400, 511, 512, 700], [2], [899]])
def test_prompt_values_outside_the_window_hold_anything(q_, dim, bad, at):
    """A non-finite value makes its column non-finite in the rows that attend to it, and nothing else."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, window, sinks = 900, 150, 5
    q, k, v = _rows(n, 2, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    clean = v.clone()
    for a in at:
        v[a, 0, a % dim] = bad
        clean[a, 0, a % dim] = 0
    out, lse = _prompt(q_, q, k, v, [0, n], window, sinks, 0.1)
    place = torch.arange(n, device="cuda")
    keep = window_keep(place, place, window, sinks)
    reached = torch.zeros((n, dim), dtype=torch.bool, device="cuda")
    for a in at:
        reached[:, a % dim] |= keep[:, a]
    assert reached.any() and not reached.all()
    for h in range(2):
        o, l, to, tl = masked64(q[:, h], k[:, 0], clean[:, 0], 0.1, keep, "bf16")
        assert not torch.isfinite(out[:, h][reached].float()).any()
        assert_within(out[:, h][~reached], o[~reached], to[~reached])
        assert_within(lse[:, h], l, tl)


def test_prompt_rows_outside_the_window_without_sinks(q_):
    """Without sinks a bad key leaves the window, and later rows are right again."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n, window = 1000, 100
    q, k, v = _rows(n, 2, 128, g), _rows(n, 1, 128, g), _rows(n, 1, 128, g)
    k[300], v[555] = float("nan"), float("inf")
    out, lse = _prompt(q_, q, k, v, [0, n], window, 0, 0.1)
    at = torch.arange(n, device="cuda")
    keep = window_keep(at, at, window, 0)
    hit = keep[:, 300] | keep[:, 555]
    for h in range(2):
        o, l, to, tl = masked64(q[~hit, h], k[:, 0], v[:, 0], 0.1, keep[~hit], "bf16")
        assert_within(out[~hit, h], o, to)
        assert_within(lse[~hit, h], l, tl)
    assert not torch.isfinite(out[hit].float()).any()


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_query_tiles_without_rows_do_not_run_ahead(q_, dim):
    """Blocks of one query tile among blocks of two, many items a CTA, with NaN left in shared memory: a warp that
    looks through values which have not arrived yet spoils them."""
    g = torch.Generator(device="cuda").manual_seed(12)
    lens = [100, 3001, 600, 128, 700, 1100, 64, 2500, 333, 900]
    heads, hk, t = 28, 4, sum(lens)
    q, k, v = _rows(t, heads, dim, g, 1.5), _rows(t, hk, dim, g), _rows(t, hk, dim, g)
    cu = _offsets(lens)
    poison = torch.full_like(v, float("nan"))
    dev_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for window, sinks in ((500, 4), (100, 0), (1000, 130)):
        q_.prompt_attention(q, k, poison, dev_cu, 0.1)
        out, lse = _prompt(q_, q, k, v, cu, window, sinks, 0.1)
        for i in range(len(lens)):
            rows, at = slice(cu[i], cu[i + 1]), torch.arange(lens[i], device="cuda")
            keep = window_keep(at, at, window, sinks)
            for h in range(heads):
                o, l, to, tl = masked64(q[rows, h], k[rows, h // 7], v[rows, h // 7], 0.1, keep, "bf16")
                assert_within(out[rows, h], o, to, f"window {window} sequence {i} head {h}")


def test_prompt_window_without_effect_is_the_plain_call(q_):
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = _rows(700, 4, 128, g), _rows(700, 2, 128, g), _rows(700, 2, 128, g)
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    want = q_.prompt_attention(q, k, v, cu, 0.1)
    got = q_.window_prompt_attention(q, k, v, cu, 700, 0, 0.1)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for window, sinks in ((400, 3), (1, 700)):  # of the rows, not of a sequence: the weights round otherwise
        got = q_.window_prompt_attention(q, k, v, cu, window, sinks, 0.1)
        _check_prompt(q, k, v, [0, 300, 700], window, sinks, 0.1, *got)
        _check_prompt(q, k, v, [0, 300, 700], 700, 0, 0.1, *got)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_scores_of_any_size(q_, dim):
    """Scores up to 1e32: the largest visible key has all of the weight, and nothing is lost to the reference."""
    g = torch.Generator(device="cuda").manual_seed(15)
    n, window, sinks = 400, 100, 3
    q, k, v = _rows(n, 2, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    for size in (1e9, 1e12, 1e30):
        big = q * size
        out, lse = _prompt(q_, big, k, v, [0, n], window, sinks, 1.0)
        at = torch.arange(n, device="cuda")
        keep = window_keep(at, at, window, sinks)
        for h in range(2):
            score = torch.where(keep, big[:, h].double() @ k[:, 0].double().T, -math.inf)
            top2 = score.topk(2, 1).values
            # fp32 products and sums: 2^-20 of the magnitudes (attention_reference), and 2^100 between the weights
            near = 2.0 ** -20 * (big[:, h].double().abs() @ k[:, 0].double().abs().T).amax(1)
            clear = top2[:, 0] - top2[:, 1] > 2 * near + 100
            assert clear[1:].float().mean() > 0.9
            assert torch.equal(out[clear, h].double(), v[score.argmax(1)][clear, 0].double())
            assert ((lse[:, h].double() - top2[:, 0]).abs() <= near + 2.0 ** -22 * top2[:, 0].abs() + math.log(n))[clear].all()


def test_prompt_rows_masked_by_infinite_scores(q_):
    """Every visible score -inf: zeros and -inf."""
    q, k, v = (torch.ones((300, 1, 64), dtype=BF, device="cuda") for _ in range(3))
    k[100:250] = -float("inf")
    out, lse = _prompt(q_, q, k, v, [0, 300], 20, 0, 0.1)
    assert (out[119:250] == 0).all() and (lse[119:250] == -math.inf).all()
    assert (out[:100] == 1).all() and (out[251:] == 1).all()


# ---- one new token per sequence over the paged cache --------------------------


def _cache(q_, lens, hk, dim, page, dtype, g, dropped=None):
    """Shuffled pages with NaN in every row that no sequence holds, out-of-range entries past the last page;
    dropped(i, page index): the entry of a page that is to be never read."""
    n = len(lens)
    used = [-(-m // page) for m in lens]
    order = torch.randperm(sum(used) + 1, generator=torch.Generator().manual_seed(1)).tolist()
    table = torch.full((n, max(used + [1])), 2 ** 30, dtype=torch.int32)
    raw = torch.uint8 if dtype == F8 else BF
    pages = [torch.full((sum(used) + 1, hk, page, dim), 0x7F if dtype == F8 else float("nan"), dtype=raw, device="cuda")
             for _ in range(2)]
    rows = []
    at = 0
    for i, m in enumerate(lens):
        mine = []
        for x in pages:
            r = torch.randn((hk, m, dim), generator=g, device="cuda")
            r = (r * 100).clamp(-448, 448).to(F8) if dtype == F8 else r.to(BF)
            mine.append(r)
            for j in range(used[i]):
                part = slice(j * page, min((j + 1) * page, m))
                x[order[at + j], :, :part.stop - part.start] = r[:, part].view(raw)
        for j in range(used[i]):
            table[i, j] = order[at + j]
            if dropped is not None and dropped(i, j):
                table[i, j] = -1 - j
        at += used[i]
        rows.append(mine)
    ks = vs = None
    if dtype == F8:
        ks, vs = (torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.005 for _ in range(2))
    return q_.kv_cache(pages[0].view(dtype), pages[1].view(dtype), table.cuda(), ks, vs), rows, ks, vs


def _check_decode(lens, q, rows, ks, vs, window, sinks, scale, out, lse):
    hk = rows[0][0].shape[0]
    group = q.shape[1] // hk
    for i, m in enumerate(lens):
        keep = window_keep(torch.tensor([m - 1], device="cuda"), torch.arange(m, device="cuda"), window, sinks)
        for j in range(hk):
            mine = slice(j * group, (j + 1) * group)
            k, v = (x[j].double() for x in rows[i])
            if ks is not None:
                k, v = k * ks[j].double(), v * vs[j].double()
            o, l, to, tl = masked64(q[i, mine], k, v, scale, keep.expand(group, m), "split" if ks is None else "fp16")
            assert_within(out[i, mine], o, to, f"sequence {i} head {j}")
            if m == 0:
                assert (lse[i, mine] == -math.inf).all()
            else:
                assert_within(lse[i, mine], l, tl, f"lse of sequence {i} head {j}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 4), (64, 0), (100, 4), (128, 64), (500, 129), (1000, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (5, 700)])
@pytest.mark.parametrize("heads,hk,dim,page,dtype", [(28, 4, 128, 16, BF), (40, 8, 128, 24, F8), (8, 8, 64, 1, BF),
                                                     (45, 3, 64, 100, F8), (12, 1, 128, 64, BF)])
def test_decode_windows(q_, window, sinks, heads, hk, dim, page, dtype):
    g = torch.Generator(device="cuda").manual_seed(window % 1000 + sinks % 1000 + heads)
    lens = [1, 0, 700, 64, 65, 2300, 3, 128, 500]
    cache, rows, ks, vs = _cache(q_, lens, hk, dim, page, dtype, g)
    q = _rows(len(lens), heads, dim, g, 1.5, 8)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(len(lens), heads, hk, dim))
    out, lse = q_.window_decode_attention(cache, q, lengths, window, sinks, 1 / math.sqrt(dim), ws)
    assert q_.qerl_read_status(ws) == 0
    _check_decode(lens, q, rows, ks, vs, window, sinks, 1 / math.sqrt(dim), out, lse)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_decode_never_reads_pages_outside_the_window(q_, dtype):
    """Their entries are out of range and would be recorded; their rows are NaN."""
    lens, window, sinks, page = [5000, 300, 901, 40], 256, 20, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    cache, rows, ks, vs = _cache(q_, lens, 4, 128, page, dtype, g,
                                 lambda i, j: j * page >= sinks and (j + 1) * page <= lens[i] - window)
    q = _rows(len(lens), 28, 128, g)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(len(lens), 28, 4, 128))
    out, lse = q_.window_decode_attention(cache, q, lengths, window, sinks, 0.1, ws)
    assert q_.qerl_read_status(ws) == 0
    _check_decode(lens, q, rows, ks, vs, window, sinks, 0.1, out, lse)


def test_decode_many_sequences_and_one_long(q_):
    """More sequences than threads, and one that many CTAs share, whose positions pass the window many times."""
    g = torch.Generator(device="cuda").manual_seed(9)
    lens = [int(x) for x in torch.randint(0, 400, (300,), generator=torch.Generator().manual_seed(4))]
    lens[17] = 60000
    cache, rows, ks, vs = _cache(q_, lens, 2, 64, 64, BF, g)
    q = _rows(len(lens), 10, 64, g)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for window, sinks in ((64, 4), (30000, 100)):
        out, lse = q_.window_decode_attention(cache, q, lengths, window, sinks, 0.125)
        _check_decode(lens, q, rows, ks, vs, window, sinks, 0.125, out, lse)


def test_decode_out_of_range_lengths_are_clamped_and_recorded(q_):
    g = torch.Generator(device="cuda").manual_seed(10)
    cache, rows, ks, vs = _cache(q_, [64, 64, 64], 2, 64, 16, BF, g)
    q = _rows(3, 4, 64, g)
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(3, 4, 2, 64))
    out, lse = q_.window_decode_attention(cache, q, torch.tensor([-5, 65, 2 ** 31 - 1], dtype=torch.int32, device="cuda"),
                                          20, 2, 0.1, ws)
    assert q_.STATUS_NAMES[q_.qerl_read_status(ws)] == "QERL_ERR_RANGE"
    _check_decode([0, 64, 64], q, [[x[:, :0] for x in rows[0]], rows[1], rows[2]], ks, vs, 20, 2, 0.1, out, lse)


def test_decode_graph_follows_the_lengths(q_):
    """A captured call takes the lengths that stand there when it is replayed."""
    g = torch.Generator(device="cuda").manual_seed(11)
    lens = [900, 200]
    cache, rows, ks, vs = _cache(q_, lens, 2, 128, 16, BF, g)
    q = _rows(2, 10, 128, g)
    lengths = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q).contiguous(), torch.empty((2, 10), device="cuda")
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(2, 10, 2, 128))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q_.check(q_.qerl_window_decode_attention(cache, q, lengths, 100, 4, 0.1, out, lse, ws))
    for now in ([900, 200], [104, 105], [3, 0], [500, 1]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(now, q, [[x[:, :m] for x in r] for m, r in zip(now, rows)], ks, vs, 100, 4, 0.1, out, lse)
