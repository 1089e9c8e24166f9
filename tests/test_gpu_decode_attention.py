"""Attention of one new token per sequence over the paged cache, on the GPU, against the 64-bit form."""
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


def _setup(q_, lens, heads, hk, dim, page, dtype, seed=0, pad=0, spare=2, q_std=1.5, first_page=0):
    """A cache whose rows past every length, and whose unused pages, hold NaN; page numbers shuffled;
    table entries past the last page out of range (they are never to be read)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 17)
    n = len(lens)
    used = [-(-m // page) for m in lens]
    num = sum(used) + spare
    width = max(max(used), 1)
    order = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((n, width + pad), 2 ** 30, dtype=torch.int32)
    shape = (first_page + num, hk, page, dim)
    raw = torch.uint8 if dtype == F8 else BF
    nan_bits = 0x7F if dtype == F8 else float("nan")
    kp, vp = (torch.full(shape, nan_bits, dtype=raw, device="cuda") for _ in range(2))
    rows = []
    at = 0
    for i, m in enumerate(lens):
        k = torch.randn((hk, m, dim), generator=g, device="cuda")
        v = torch.randn((hk, m, dim), generator=g, device="cuda") + 0.25
        if dtype == F8:
            k, v = (k * 100).clamp(-448, 448).to(F8), (v * 100).clamp(-448, 448).to(F8)  # torch's cast gives NaN past 448
        else:
            k, v = k.to(BF), v.to(BF)
        rows.append((k, v))
        for j in range(used[i]):
            p = first_page + order[at]
            at += 1
            table[i, j] = p
            part = slice(j * page, min((j + 1) * page, m))
            kp[p, :, :part.stop - part.start] = k[:, part].view(raw)
            vp[p, :, :part.stop - part.start] = v[:, part].view(raw)
    ks = vs = None
    if dtype == F8:
        ks = torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.005
        vs = torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.005
    cache = q_.kv_cache(kp.view(dtype), vp.view(dtype), table.cuda()[:, :width], ks, vs)
    full = torch.full((n, heads * dim + 8 * pad), float("nan"), dtype=BF, device="cuda")
    full[:, :heads * dim] = (torch.randn((n, heads * dim), generator=g, device="cuda") * q_std).to(BF)
    q = full[:, :heads * dim].unflatten(1, (heads, dim))
    return cache, q, rows, ks, vs


def _check(lens, q, rows, ks, vs, scale, out, lse, what=""):
    heads, hk = q.shape[1], rows[0][0].shape[0]
    group = heads // hk
    for i in range(len(lens)):
        for j in range(hk):
            mine = slice(j * group, (j + 1) * group)
            k, v = (x[j].double() for x in rows[i])
            if ks is not None:
                k, v = k * ks[j].double(), v * vs[j].double()
            o, l, to, tl = attend64(q[i, mine], k, v, scale, "split" if ks is None else "fp16")
            assert_within(out[i, mine], o, to, f"{what} sequence {i} head {j}")
            if lens[i] == 0:
                assert (lse[i, mine] == -math.inf).all()
            else:
                assert_within(lse[i, mine], l, tl, f"{what} lse of sequence {i} head {j}")


def _run(q_, cache, q, lens, scale, ws=None, stream=None, pad=0):
    n, h, d = q.shape
    out = torch.full((n, h * d + 8 * pad), float("nan"), dtype=BF, device="cuda")[:, :h * d].unflatten(1, (h, d))
    lse = torch.full((n, h), float("nan"), device="cuda")
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(n, h, cache.num_kv_heads, d)) if ws is None else ws
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()
    q_.check(q_.qerl_decode_attention(cache, q, lengths, scale, out, lse, ws, stream=stream))
    assert q_.qerl_read_status(ws, stream=stream) == 0
    return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 0, 127, 128, 129, 300, 1000, 0]


@pytest.mark.parametrize("heads,hk,dim", [(28, 4, 128), (16, 2, 128), (40, 8, 64), (3, 3, 64), (12, 1, 128),
                                          (45, 3, 64), (17, 1, 64), (40, 1, 128)])
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("page", [1, 16, 24, 128])
def test_lengths_pages_and_groups(q_, heads, hk, dim, dtype, page):
    cache, q, rows, ks, vs = _setup(q_, EDGES, heads, hk, dim, page, dtype, pad=3)
    scale = 1 / math.sqrt(dim)
    out, lse = _run(q_, cache, q, EDGES, scale, pad=2)
    _check(EDGES, q, rows, ks, vs, scale, out, lse)


@pytest.mark.parametrize("lens", [[1], [64], [777], [30011], [5, 30011, 1], [4097] * 40, [0, 0, 0], [0, 9, 0]])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_splits_and_joins(q_, lens, dtype):
    """One sequence over all CTAs, many over few, a stretch that begins and ends inside sequences; the
    workspace is used again at once, and the result is the same bit for bit."""
    heads, hk, dim, page = 28, 4, 128, 32
    cache, q, rows, ks, vs = _setup(q_, lens, heads, hk, dim, page, dtype, seed=len(lens))
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(len(lens), heads, hk, dim))
    scale = 1 / math.sqrt(dim)
    out, lse = _run(q_, cache, q, lens, scale, ws=ws)
    _check(lens, q, rows, ks, vs, scale, out, lse)
    for _ in range(3):
        again, lse2 = _run(q_, cache, q, lens, scale, ws=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_many_sequences(q_):
    """More sequences than a CTA has threads, most of them empty or short."""
    lens = [(i * 7919) % 41 if i % 3 else 0 for i in range(700)]
    cache, q, rows, ks, vs = _setup(q_, lens, 8, 2, 64, 8, BF)
    out, lse = _run(q_, cache, q, lens, 0.125)
    _check(lens, q, rows, ks, vs, 0.125, out, lse)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_flat_negative_and_peaked_scores(q_, dtype, scale):
    """scale 3 with large q: the running reference moves often and most weights vanish."""
    lens = [500, 129]
    cache, q, rows, ks, vs = _setup(q_, lens, 16, 2, 128, 16, dtype, q_std=4.0)
    out, lse = _run(q_, cache, q, lens, scale)
    _check(lens, q, rows, ks, vs, scale, out, lse)


def test_growing_scores(q_):
    """Keys whose scores rise along the sequence: every step moves the reference."""
    dim, n = 64, 2000
    k = torch.zeros((1, n, dim), device="cuda")
    k[0, :, 0] = torch.arange(n, device="cuda") * 0.5
    k = k.to(BF)
    v = torch.randn((1, n, dim), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(BF)
    q = torch.zeros((1, 1, dim), device="cuda", dtype=BF)
    q[0, 0, 0] = 1.0
    table = torch.arange(n // 8, dtype=torch.int32, device="cuda")[None]
    paged = lambda x: x.view(1, n // 8, 8, dim).transpose(0, 1).contiguous()
    for sign in (1.0, -1.0):
        out, lse = _run(q_, q_.kv_cache(paged(k), paged(v), table), q, [n], sign)
        _check([n], q, [(k, v)], None, None, sign, out, lse)


@pytest.mark.parametrize("q_std", [1e-30, 1e30])
def test_extreme_query_scales_over_an_8_bit_cache(q_, q_std):
    lens = [200]
    cache, q, rows, ks, vs = _setup(q_, lens, 8, 2, 64, 16, F8, q_std=q_std)
    scale = 0.1 / q_std
    out, lse = _run(q_, cache, q, lens, scale)
    _check(lens, q, rows, ks, vs, scale, out, lse)


def test_non_finite_values_in_use(q_):
    """A NaN in a used key or value reaches its sequence's head alone; infinite scores of every key
    (all -inf) give the empty row."""
    lens = [70, 70, 70]
    cache, q, rows, ks, vs = _setup(q_, lens, 4, 2, 64, 16, BF)
    kp, vp, table = cache.tensors[0], cache.tensors[1], cache.tensors[2]
    kp[table[0, 1].item(), 0, 3, 5] = float("nan")
    vp[table[1, 2].item(), 1, 7, 9] = float("nan")
    q[2] = 0
    q[2, :, 0] = 1.0
    for j in range(5):
        rows_in = min(16, 70 - 16 * j)
        kp[table[2, j].item(), 0, :rows_in, 0] = -float("inf")
    n, h, d = q.shape
    out, lse = _run(q_, cache, q, lens, 0.125)
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isfinite(out[0, 2:]).all() and torch.isfinite(out[1, :2]).all()
    assert torch.isnan(out[1, 2:, 9]).all()
    assert torch.isfinite(out[1, 2:, [c for c in range(d) if c != 9]]).all()
    assert (out[2, :2] == 0).all() and (lse[2, :2] == -math.inf).all()
    assert torch.isfinite(out[2, 2:]).all()


def test_offsets_past_32_bits(q_):
    """Pages past 4 GB of each tensor."""
    lens, page, hk, dim = [130, 64], 64, 8, 128
    first = (2 ** 32 + 2 ** 20) // (page * hk * dim * 2)
    cache, q, rows, ks, vs = _setup(q_, lens, 40, hk, dim, page, BF, first_page=first)
    out, lse = _run(q_, cache, q, lens, 0.09)
    _check(lens, q, rows, ks, vs, 0.09, out, lse)
    # and the append of one more token there
    g = torch.Generator(device="cuda").manual_seed(1)
    new = torch.randn((2, hk, dim), generator=g, device="cuda").to(BF)
    ws = q_.workspace(q_.qerl_rope_append_workspace_size())
    pos = torch.tensor([130, 63], dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_rope_append(cache, None, new, new, pos, torch.empty(0, dtype=torch.float64, device="cuda"), None,
                                 None, ws))
    assert q_.qerl_read_status(ws) == 0
    kp, table = cache.tensors[0], cache.tensors[2]
    assert torch.equal(kp[table[0, 2].item(), :, 2], new[0]) and torch.equal(kp[table[1, 0].item(), :, 63], new[1])


def test_stream_and_graph(q_):
    lens = [700, 3, 1200]
    cache, q, rows, ks, vs = _setup(q_, lens, 28, 4, 128, 16, BF)
    scale = 0.09
    a, la = _run(q_, cache, q, lens, scale)
    b, lb = _run(q_, cache, q, lens, scale, stream=torch.cuda.Stream())
    assert torch.equal(a, b) and torch.equal(la, lb)
    n, h, d = q.shape
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(n, h, 4, d))
    out, lse = torch.zeros_like(a), torch.zeros_like(la)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q_.check(q_.qerl_decode_attention(cache, q, lengths, scale, out, lse, ws))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
    lengths.copy_(torch.tensor([1, 3, 800], dtype=torch.int32))  # the lengths are read on the device
    graph.replay()
    torch.cuda.synchronize()
    short = [1, 3, 800]
    _check(short, q, [(k[:, :m], v[:, :m]) for (k, v), m in zip(rows, short)], ks, vs, scale, out, lse)


def test_bad_pages_and_lengths_are_recorded(q_):
    """Page numbers outside the cache and lengths outside the table: recorded, bounded, and the other
    sequences are right."""
    lens = [40, 40, 40, 40]
    cache, q, rows, ks, vs = _setup(q_, lens, 8, 2, 64, 16, BF)
    table = cache.tensors[2]
    n, h, d = q.shape
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(n, h, 2, d))
    out, lse = torch.empty_like(q), torch.empty((n, h), device="cuda")
    for bad, lengths in ((-1, lens), (2 ** 31 - 1, lens), (None, [40, -7, 40, 40]), (None, [40, 49, 40, 40])):
        keep = table[1, 1].item()
        if bad is not None:
            table[1, 1] = bad
        lt = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        q_.check(q_.qerl_decode_attention(cache, q, lt, 0.125, out, lse, ws))
        assert q_.STATUS_NAMES[q_.qerl_read_status(ws)] == "QERL_ERR_RANGE"
        assert q_.qerl_read_status(ws) == 0
        table[1, 1] = keep
        ok = [0, 2, 3]
        _check([40] * 3, q[ok], [rows[i] for i in ok], ks, vs, 0.125, out[ok], lse[ok])
        if lengths[1] < 0:
            assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_one_workspace_for_many_shapes(q_):
    """Calls of different shapes take turns on one workspace, which is zero-filled once."""
    shapes = [([900, 3, 77], 28, 4, 128, F8), ([5000], 12, 1, 128, BF), ([40] * 300, 8, 2, 64, BF),
              ([1, 2000], 45, 3, 64, BF)]
    need = max(q_.qerl_decode_attention_workspace_size(len(l), h, hk, d) for l, h, hk, d, _ in shapes)
    ws = q_.workspace(need)
    made = [_setup(q_, l, h, hk, d, 16, t, seed=i) for i, (l, h, hk, d, t) in enumerate(shapes)]
    for _ in range(2):
        for (lens, *_rest), (cache, q, rows, ks, vs) in zip(shapes, made):
            out, lse = _run(q_, cache, q, lens, 0.1, ws=ws)
            _check(lens, q, rows, ks, vs, 0.1, out, lse)


def test_a_table_whose_rows_overlap_is_refused(q_):
    cache, q, *_ = _setup(q_, [20, 20], 8, 2, 64, 16, BF)
    shared = q_.kv_cache(cache.tensors[0], cache.tensors[1], cache.tensors[2][:1].expand(2, -1))
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(2, 8, 2, 64))
    st = q_.qerl_decode_attention(shared, q, torch.ones(2, dtype=torch.int32, device="cuda"), 0.1, torch.empty_like(q),
                                  None, ws)
    assert q_.STATUS_NAMES[st] == "QERL_ERR_INVALID_ARGUMENT"


def test_no_lse_and_no_pages(q_):
    """lse may be left out; a cache without pages or table columns gives empty rows."""
    cache, q, rows, ks, vs = _setup(q_, [50, 300], 8, 2, 64, 16, BF)
    out, lse = _run(q_, cache, q, [50, 300], 0.1)
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(2, 8, 2, 64))
    again = torch.empty_like(out)
    lengths = torch.tensor([50, 300], dtype=torch.int32, device="cuda")
    q_.check(q_.qerl_decode_attention(cache, q, lengths, 0.1, again, None, ws))
    assert q_.qerl_read_status(ws) == 0 and torch.equal(out, again)
    none = torch.empty((0, 2, 16, 64), dtype=BF, device="cuda")
    empty = q_.kv_cache(none, none, torch.zeros((2, 0), dtype=torch.int32, device="cuda"))
    q_.check(q_.qerl_decode_attention(empty, q, lengths * 0, 0.1, out, lse, ws))
    assert q_.qerl_read_status(ws) == 0 and (out == 0).all() and (lse == -math.inf).all()


def test_binding_refuses_what_the_library_cannot_see(q_):
    """Types, shapes and strides that a raw pointer does not tell."""
    cache, q, *_ = _setup(q_, [20, 20], 8, 2, 64, 16, BF)
    n, h, d = q.shape
    ws = q_.workspace(q_.qerl_decode_attention_workspace_size(n, h, 2, d))
    good = dict(q=q, lengths=torch.tensor([20, 20], dtype=torch.int32, device="cuda"), out=torch.empty_like(q),
                lse=torch.empty((n, h), device="cuda"))
    call = lambda **kw: q_.qerl_decode_attention(cache, scale=0.1, workspace=ws, **{**good, **kw})
    assert call() == 0
    for kw, error in [(dict(q=q.float()), TypeError), (dict(out=good["out"].half()), TypeError),
                      (dict(lengths=good["lengths"].long()), TypeError), (dict(lengths=good["lengths"].cpu()), TypeError),
                      (dict(lse=good["lse"].double()), TypeError), (dict(lengths=good["lengths"][:1]), ValueError),
                      (dict(q=q[:1]), ValueError), (dict(out=good["out"][:, :4]), ValueError),
                      (dict(lse=torch.empty((h, n), device="cuda")), ValueError),
                      (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                      (dict(lengths=torch.zeros(4, dtype=torch.int32, device="cuda")[::2]), ValueError)]:
        with pytest.raises(error):
            call(**kw)
    k, v, table = cache.tensors[:3]
    for args, error in [((k.float(), v.float(), table), TypeError), ((k, v, table.long()), TypeError),
                        ((k, v[:-1], table), ValueError), ((k.transpose(1, 2), v.transpose(1, 2), table), ValueError),
                        ((k, v.view(torch.int16), table), TypeError), ((k, v, table.T.contiguous().T), ValueError),
                        ((k.view(torch.uint8)[..., :64].contiguous().view(F8), v.view(torch.uint8)[..., :64].contiguous()
                          .view(F8), table, torch.ones(3, device="cuda")), ValueError)]:
        with pytest.raises(error):
            q_.kv_cache(*args)
