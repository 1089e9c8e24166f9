"""Attention of drafted tokens over the paged cache and one another, on the GPU, against the 64-bit form."""
import math
import random

import pytest
import torch

from attention_reference import assert_within
from masked_reference import masked64

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Sequences of `lens` rows in the cache and `counts` new tokens.  Shuffled pages with NaN in every row that no
    sequence holds, out-of-range entries past the last page.  kind: "chain" (no mask), "tree", "any" (random bits,
    some rows without any)."""

    def __init__(self, q_, lens, counts, heads, hk, dim, page=16, dtype=BF, kind="tree", seed=0, pad=0, lead=0, tail=0,
                 q_std=1.5, words=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = random.Random(seed)
        n = len(lens)
        self.q_, self.lens, self.counts, self.heads, self.hk, self.dim = q_, lens, counts, heads, hk, dim
        used = [-(-m // page) for m in lens]
        order = r.sample(range(sum(used) + 1), sum(used) + 1)
        table = torch.full((n, max(used + [1]) + pad), 2 ** 30, dtype=torch.int32)
        raw = torch.uint8 if dtype == F8 else BF
        pages = [torch.full((sum(used) + 1, hk, page, dim), 0x7F if dtype == F8 else float("nan"), dtype=raw,
                            device="cuda") for _ in range(2)]
        self.rows, at = [], 0
        for i, m in enumerate(lens):
            mine = []
            for x in pages:
                y = torch.randn((hk, m, dim), generator=g, device="cuda")
                y = (y * 100).clamp(-448, 448).to(F8) if dtype == F8 else y.to(BF)
                mine.append(y)
                for j in range(used[i]):
                    part = slice(j * page, min((j + 1) * page, m))
                    x[order[at + j], :, :part.stop - part.start] = y[:, part].view(raw)
            table[i, :used[i]] = torch.tensor(order[at:at + used[i]], dtype=torch.int32)
            at += used[i]
            self.rows.append(mine)
        self.ks = self.vs = None
        if dtype == F8:
            self.ks, self.vs = (torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.005 for _ in range(2))
        self.pages, self.raw = pages, raw
        self.cache = q_.kv_cache(pages[0].view(dtype), pages[1].view(dtype), table.cuda()[:, :max(used + [1])], self.ks,
                                 self.vs)
        self.cu = [lead]
        for c in counts:
            self.cu.append(self.cu[-1] + c)
        self.tokens = self.cu[-1] + tail
        self.q = _rows(self.tokens, heads, dim, g, q_std, pad * 8)
        self.k, self.v = _rows(self.tokens, hk, dim, g, 1.0, pad * 16), _rows(self.tokens, hk, dim, g, 1.0, pad * 24)
        self.keep, self.mask = [], None
        words = words or max(1, -(-max(counts + [1]) // 64))
        bits = torch.zeros((self.tokens, words), dtype=torch.int64)
        for s, c in enumerate(counts):
            seen = []
            for t in range(c):
                if kind == "chain":
                    seen.append((2 << t) - 1)
                elif kind == "tree":
                    parent = r.randint(max(-1, t - 6), t - 1)
                    seen.append((seen[parent] if parent >= 0 else 0) | 1 << t)
                else:
                    seen.append(0 if r.random() < 0.2 else r.getrandbits(c))
                junk = r.getrandbits(64 * words) >> c << c  # bits past the sequence's tokens
                for w in range(words):
                    word = ((seen[-1] | junk) >> (64 * w)) & (2 ** 64 - 1)
                    bits[self.cu[s] + t, w] = word - 2 ** 64 if word >= 2 ** 63 else word
            self.keep.append(torch.tensor([[bool(x >> j & 1) for j in range(c)] for x in seen]).reshape(c, c).cuda())
        if kind != "chain":
            self.mask = bits.cuda()

    def run(self, scale, ws=None, stream=None, status="QERL_OK", pad=0):
        shape = (self.tokens, self.heads * self.dim + pad)
        out = torch.full(shape, 5.0, dtype=BF, device="cuda")[:, :self.heads * self.dim].unflatten(1, (self.heads, self.dim))
        lse = torch.full((self.tokens, self.heads), 5.0, device="cuda")
        if ws is None:
            ws = self.workspace()
        cu, lengths = _i32(self.cu), _i32(self.lens)
        torch.cuda.synchronize()
        self.q_.check(self.q_.qerl_tree_attention(self.cache, self.q, self.k, self.v, cu, lengths, self.mask, scale, out, lse,
                                                  ws, stream=stream))
        assert self.q_.STATUS_NAMES[self.q_.qerl_read_status(ws, stream=stream)] == status
        return out, lse

    def workspace(self):
        ws = self.q_.workspace(self.q_.qerl_tree_attention_workspace_size(self.tokens, self.heads, self.hk, self.dim,
                                                                          len(self.lens)))
        ws[256:] = 0xFF  # only the header is zero-filled: floats of NaN
        return ws

    def check(self, scale, out, lse, what=""):
        group = self.heads // self.hk
        for s, (m, c) in enumerate(zip(self.lens, self.counts)):
            rows = slice(self.cu[s], self.cu[s] + c)
            if c == 0:
                continue
            keep = torch.cat([torch.ones((c, m), dtype=torch.bool, device="cuda"), self.keep[s]], 1)
            for h in range(self.heads):
                j = h // group
                k, v = (x[j].double() for x in self.rows[s])
                if self.ks is not None:
                    k, v = k * self.ks[j].double(), v * self.vs[j].double()
                k, v = torch.cat([k, self.k[rows, j].double()]), torch.cat([v, self.v[rows, j].double()])
                o, l, to, tl = masked64(self.q[rows, h], k, v, scale, keep, "bf16")
                assert_within(out[rows, h], o, to, f"{what} sequence {s} head {h}")
                none = torch.isinf(l)
                assert (lse[rows, h][none] == -math.inf).all() and (out[rows, h][none] == 0).all()
                assert_within(lse[rows, h][~none], l[~none], tl[~none], f"{what} lse of sequence {s} head {h}")


BLOCKS = [(28, 4, 128, 16, BF), (40, 8, 128, 24, F8), (8, 8, 64, 1, BF), (45, 3, 64, 100, F8), (12, 1, 128, 64, F8),
          (10, 2, 64, 32, BF)]


@pytest.mark.parametrize("heads,hk,dim,page,dtype", BLOCKS)
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
def test_one_sequence(q_, heads, hk, dim, page, dtype, kind):
    for m, c in ((0, 1), (1, 1), (127, 3), (128, 5), (300, 17), (1000, 64)):
        case = Case(q_, [m], [c], heads, hk, dim, page, dtype, kind, seed=m + c)
        out, lse = case.run(1 / math.sqrt(dim))
        case.check(1 / math.sqrt(dim), out, lse, f"{m} + {c}")


@pytest.mark.parametrize("heads,hk,dim,page,dtype", BLOCKS)
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
def test_ragged_batches(q_, heads, hk, dim, page, dtype, kind):
    """Empty caches, sequences without new tokens, segments of one, two and more query tiles."""
    lens = [5, 0, 700, 128, 129, 2000, 0, 383, 64]
    counts = [3, 7, 0, 33, 16, 50, 61, 1, 25]
    case = Case(q_, lens, counts, heads, hk, dim, page, dtype, kind, seed=heads, pad=1, lead=4, tail=9)
    out, lse = case.run(1 / math.sqrt(dim), pad=24)
    case.check(1 / math.sqrt(dim), out, lse)
    for x in (out, lse):  # rows of no sequence
        assert (x[:4] == 5).all() and (x[-9:] == 5).all()
    again, lse2 = case.run(1 / math.sqrt(dim), stream=torch.cuda.Stream())
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("counts", [[130], [64, 65, 128, 129], [300, 1, 256]])
def test_more_new_tokens_than_a_key_tile(q_, kind, dtype, counts):
    case = Case(q_, [200 + 100 * i for i in range(len(counts))], counts, 8, 2, 64, 16, dtype, kind, seed=sum(counts))
    out, lse = case.run(0.125)
    case.check(0.125, out, lse)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("count", [2, 40])
def test_one_long_sequence(q_, dtype, count):
    """Every CTA has a part of every head, joined in CTA order."""
    case = Case(q_, [30011], [count], 14, 2, 128, 64, dtype, "tree", seed=3)
    out, lse = case.run(0.09)
    case.check(0.09, out, lse)


@pytest.mark.parametrize("heads,hk", [(1, 1), (64, 1), (200, 1)])
def test_group_sizes(q_, heads, hk):
    case = Case(q_, [500, 30], [9, 2], heads, hk, 64, 16, BF, "tree", seed=heads)
    out, lse = case.run(0.125)
    case.check(0.125, out, lse)


def test_more_sequences_than_threads(q_):
    r = random.Random(2)
    n = 1300
    lens = [r.choice([0, 3, 40]) for _ in range(n)]
    counts = [r.choice([0, 0, 1, 2]) for _ in range(n)]
    lens[900], counts[900], counts[0], counts[-1] = 9000, 5, 0, 0
    case = Case(q_, lens, counts, 4, 2, 64, 16, BF, "chain", seed=5)
    out, lse = case.run(0.125)
    case.check(0.125, out, lse)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.2, 1.0), (2.0, 3.0), (0.5, 8.0)])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_flat_negative_and_peaked_scores(q_, scale, std, dtype):
    case = Case(q_, [700, 90], [12, 30], 8, 2, 128, 16, dtype, "tree", seed=4, q_std=std)
    out, lse = case.run(scale)
    case.check(scale, out, lse)


def test_negative_key_scale(q_):
    case = Case(q_, [300], [6], 4, 2, 64, 16, F8, "tree", seed=6)
    case.ks.neg_()
    out, lse = case.run(0.2)
    case.check(0.2, out, lse)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("count", [3, 200])
def test_growing_scores(q_, sign, count):
    """Scores that rise along the keys: the reference moves in every tile and O is rescaled."""
    case = Case(q_, [1500], [count], 2, 1, 64, 16, BF, "chain", seed=7)
    case.q.zero_()
    case.q[:, :, 0] = 1.0
    ramp = (torch.arange(1500, device="cuda") * 0.25).to(BF)
    case.rows[0][0].zero_()
    case.rows[0][0][0, :, 0] = ramp
    table = case.cache.tensors[2][0].long()
    case.pages[0][table[torch.arange(1500, device="cuda") // 16], 0, torch.arange(1500, device="cuda") % 16] = \
        case.rows[0][0][0]
    case.k.zero_()
    case.k[:, 0, 0] = (400 + torch.arange(count, device="cuda")).to(BF)
    out, lse = case.run(sign)
    case.check(sign, out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("place", ["k", "v"])
@pytest.mark.parametrize("count,heads", [(20, 4), (70, 8), (140, 2)])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_new_tokens_that_are_not_seen_hold_anything(q_, bad, place, count, heads, dtype):
    """A non-finite key or value of a draft reaches the tokens that see it and no others."""
    case = Case(q_, [200, 77], [count, 5], heads, 2, 64, 16, dtype, "any", seed=8)
    at = [0, 3, count - 1]
    x = {"k": case.k, "v": case.v}[place]
    for a in at:
        x[a, :, a % 64] = bad
    out, lse = case.run(0.1)
    hit = case.keep[0][:, at].any(1)
    assert hit.any() and not hit.all()
    safe = torch.ones(case.tokens, dtype=torch.bool, device="cuda")
    safe[:count] = ~hit
    for a in at:
        x[a, :, a % 64] = 0
    clean, lse2 = case.run(0.1)
    case.check(0.1, clean, lse2)
    assert torch.equal(out[safe], clean[safe]) and torch.equal(lse[safe], lse2[safe])
    if place == "v":
        assert torch.equal(lse, lse2)
        for a in at:
            reached = case.keep[0][:, a].nonzero()[:, 0]
            assert not torch.isfinite(out[reached, :, a % 64].float()).any()
        rest = [c for c in range(64) if c not in {a % 64 for a in at}]
        assert torch.equal(out[:, :, rest], clean[:, :, rest])
    else:  # a score of -inf has weight 0, any other that is not finite is seen in the output
        for a in at:
            score = case.q[:count, :, a % 64].float() * bad
            reached = case.keep[0][:, a][:, None] & (score != -math.inf)
            assert not torch.isfinite(out[:count][reached].float()).any()


def test_non_finite_cache_rows_reach_the_outputs(q_):
    """A key that is NaN, a value that is NaN (E4M3) or infinite (bf16): tokens of that sequence alone."""
    for dtype in (BF, F8):
        for which in (0, 1):
            case = Case(q_, [300, 300], [5, 5], 4, 2, 128, 16, dtype, "tree", seed=9)
            want, _ = case.run(0.1)
            p = int(case.cache.tensors[2][0, 7])
            case.pages[which][p, :, 3, 40] = 0xFF if dtype == F8 else float("inf" if which else "nan")
            out, lse = case.run(0.1)
            assert not torch.isfinite(out[:5, :, 40 if which else slice(None)].float()).any()
            assert torch.equal(out[5:], want[5:])


def test_every_e4m3_value(q_):
    """One key per sequence: the output is its value, which passes exactly."""
    codes = [c for c in range(256) if c & 0x7F != 0x7F]
    case = Case(q_, [1] * 4, [1] * 4, 1, 1, 64, 4, F8, "any", seed=1)
    case.mask.zero_()
    case.vs.fill_(1.0)
    table = case.cache.tensors[2]
    values = torch.tensor((codes + [0, 0])[:256], dtype=torch.uint8, device="cuda").view(4, 64)
    for s in range(4):
        case.pages[1][int(table[s, 0]), 0, 0] = values[s]
    out, _ = case.run(0.1)
    assert torch.equal(out[:, 0].float(), values.view(F8).float())


@pytest.mark.parametrize("offsets", [[0, 60, 40, 100], [0, 100, 0, 100], [0, 50, 101, 101], [-1, 50, 100, 100],
                                     [10, 5, 20, 100]])
def test_broken_offsets_leave_every_row_alone(q_, offsets):
    case = Case(q_, [20, 30, 40], [50, 25, 25], 4, 2, 64, 16, BF, "chain", seed=1)
    good = case.cu
    case.cu = offsets
    out, lse = case.run(0.1, status="QERL_ERR_RANGE")
    assert (out == 5).all() and (lse == 5).all()
    case.cu = good
    out, lse = case.run(0.1)
    case.check(0.1, out, lse)


def test_lengths_and_pages_outside_are_recorded(q_):
    case = Case(q_, [64, 64, 64], [4, 4, 4], 4, 2, 64, 16, BF, "tree", seed=1)
    case.lens = [-5, 65, 2 ** 31 - 1]
    out, lse = case.run(0.1, status="QERL_ERR_RANGE")
    case.lens = [0, 64, 64]
    case.rows[0] = [x[:, :0] for x in case.rows[0]]
    case.check(0.1, out, lse)
    # a page outside the cache: its rows read as zeros
    for number in (-1, 10 ** 6):
        case = Case(q_, [64], [4], 4, 2, 64, 16, BF, "tree", seed=1)
        case.cache.tensors[2][0, 2] = number
        for x in case.rows[0]:
            x[:, 32:48] = 0
        out, lse = case.run(0.1, status="QERL_ERR_RANGE")
        case.check(0.1, out, lse)


def test_tokens_past_the_mask_are_seen_by_none(q_):
    case = Case(q_, [100, 10], [70, 3], 4, 2, 64, 16, BF, "any", seed=2, words=1)
    case.keep[0][:, 64:] = False
    out, lse = case.run(0.1, status="QERL_ERR_RANGE")
    case.check(0.1, out, lse)


def test_one_workspace_for_ordered_calls_of_many_shapes(q_):
    shapes = [([3000], [9], 28, 4, 128), ([40, 900, 7], [60, 2, 31], 8, 8, 64), ([0], [1], 12, 1, 128)]
    cases = [Case(q_, lens, counts, h, hk, d, 16, BF, "tree", seed=i) for i, (lens, counts, h, hk, d) in enumerate(shapes)]
    ws = q_.workspace(max(c.workspace().numel() for c in cases))
    for _ in range(2):
        for c in cases:
            out, lse = c.run(0.1, ws=ws)
            c.check(0.1, out, lse)


def test_captured_calls_follow_lengths_and_masks(q_):
    """A replay takes the lengths, offsets and masks that stand there; two graphs in order share a workspace."""
    case = Case(q_, [900, 200], [20, 30], 10, 2, 128, 16, BF, "tree", seed=11)
    lens, cu, lengths = list(case.lens), _i32(case.cu), _i32(case.lens)
    out, lse = torch.empty((50, 10, 128), dtype=BF, device="cuda"), torch.empty((50, 10), device="cuda")
    ws = case.workspace()
    graphs = []
    for _ in range(2):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q_.check(q_.qerl_tree_attention(case.cache, case.q, case.k, case.v, cu, lengths, case.mask, 0.1, out, lse, ws))
        graphs.append(graph)
    rows = case.rows
    for now, counts in (([900, 200], [20, 30]), ([0, 200], [1, 49]), ([899, 1], [50, 0]), ([128, 129], [25, 25])):
        lengths.copy_(_i32(now))
        case.lens, case.counts, case.cu = now, counts, [0, counts[0], 50]
        case.rows = [[x[:, :m] for x in r] for m, r in zip(now, rows)]
        case.keep = [torch.ones((c, c), dtype=torch.bool, device="cuda").tril() for c in counts]
        cu.copy_(_i32(case.cu))
        case.mask.copy_(torch.cat([(2 << torch.arange(c)) - 1 for c in counts])[:, None])
        for graph in graphs:
            out.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            case.check(0.1, out, lse)
    assert q_.qerl_read_status(ws) == 0


def test_a_verified_draft_is_appended(q_):
    """Drafts rotated, verified and, where accepted, appended: the next token's attention over the cache is that of
    the whole sequence."""
    heads, hk, dim, page, n = 8, 2, 128, 16, 3
    lens, count = [50, 16, 0], 6
    case = Case(q_, [m + 20 for m in lens], [count] * n, heads, hk, dim, page, BF, "tree", seed=21)
    case.lens, case.rows = lens, [[x[:, :m] for x in r] for m, r in zip(lens, case.rows)]
    inv_freq = 1e4 ** (-torch.arange(dim // 2, dtype=torch.float64, device="cuda") / (dim // 2))
    depth = torch.cat([k.sum(1) for k in case.keep]).to(torch.int32) - 1
    start = torch.repeat_interleave(_i32(lens), count)
    case.q, case.k = q_.rope_append(None, case.q, case.k, None, start + depth, inv_freq)
    out, lse = case.run(0.1)
    case.check(0.1, out, lse)
    # the last token's branch of each tree is accepted
    path = torch.cat([k[-1] for k in case.keep])
    positions = torch.where(path, start + depth, -1).to(torch.int32)
    seq = torch.repeat_interleave(_i32(list(range(n))), count)
    none = torch.empty(0, dtype=torch.float64, device="cuda")
    q_.rope_append(case.cache, None, case.k, case.v, positions, none, seq_ids=seq)
    last = torch.arange(1, n + 1, device="cuda") * count - 1
    grown = (start + depth)[last] + 1
    one, lse1 = q_.decode_attention(case.cache, case.q[last].contiguous(), grown, 0.1)
    # both see the same keys; the tree's softmax weights are bf16 (2^-8), the decode's are exact to 2^-16
    for s in range(n):
        rows = slice(s * count, (s + 1) * count)
        keep = torch.cat([torch.ones(lens[s], dtype=torch.bool, device="cuda"), case.keep[s][-1]])[None]
        for h in range(heads):
            k, v = (torch.cat([a[h // 4].double(), b[rows, h // 4].double()]) for a, b in
                    zip(case.rows[s], (case.k, case.v)))
            o, l, to, tl = masked64(case.q[last[s], h][None], k, v, 0.1, keep, "split")
            assert_within(one[s, h][None], o, to)
            assert_within(lse1[s, h][None], l, tl)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_pages_past_32_bits(q_, dtype):
    """Byte offsets (and for bf16 element offsets) in the cache past 2^32."""
    case = Case(q_, [500], [7], 8, 2, 128, 16, dtype, "tree", seed=31)
    first = 2 ** 20 + 5
    far = [torch.empty((first + x.shape[0], *x.shape[1:]), dtype=x.dtype, device="cuda") for x in case.pages]
    for a, b in zip(far, case.pages):
        a[first:] = b
    assert far[0].nbytes > 2 ** 32
    table = case.cache.tensors[2]
    table += first
    case.cache = q_.kv_cache(far[0].view(dtype), far[1].view(dtype), table, case.ks, case.vs)
    out, lse = case.run(0.1)
    case.check(0.1, out, lse)


def test_two_calls_at_once(q_):
    """On two streams, each with a workspace of its own."""
    cases = [Case(q_, [3000, 20, 700], [30, 9, 61], 14, 2, 128, 16, BF, "tree", seed=41),
             Case(q_, [5000], [12], 8, 2, 64, 16, F8, "chain", seed=42)]
    streams = [torch.cuda.Stream() for _ in cases]
    made = []
    for c in cases:
        shape = (c.tokens, c.heads, c.dim)
        made.append((torch.empty(shape, dtype=BF, device="cuda"), torch.empty(shape[:2], device="cuda"), _i32(c.cu),
                     _i32(c.lens), c.workspace()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (out, lse, cu, lengths, ws), s in zip(cases, made, streams):
            q_.check(q_.qerl_tree_attention(c.cache, c.q, c.k, c.v, cu, lengths, c.mask, 0.1, out, lse, ws, stream=s))
    torch.cuda.synchronize()
    for c, (out, lse, _, _, ws) in zip(cases, made):
        assert q_.qerl_read_status(ws) == 0
        c.check(0.1, out, lse)


def test_extreme_scores_and_values(q_):
    """Queries near bf16's largest give infinite scores or weights of one key alone; nothing else is touched."""
    case = Case(q_, [200, 130], [6, 6], 4, 2, 64, 16, BF, "tree", seed=43)
    case.q[:6] *= 1e30
    out, lse = case.run(1.0)
    for s in (1,):
        rows = slice(6, 12)
        keep = torch.cat([torch.ones((6, 130), dtype=torch.bool, device="cuda"), case.keep[s]], 1)
        for h in range(4):
            k, v = (torch.cat([x[h // 2].double(), y[rows, h // 2].double()]) for x, y in zip(case.rows[s], (case.k, case.v)))
            o, l, to, tl = masked64(case.q[rows, h], k, v, 1.0, keep, "bf16")
            assert_within(out[rows, h], o, to)
            assert_within(lse[rows, h], l, tl)
    # scores up to 1e32: the largest key has all of the weight
    for h in range(4):
        keep = torch.cat([torch.ones((6, 200), dtype=torch.bool, device="cuda"), case.keep[0]], 1)
        k, v = (torch.cat([x[h // 2].double(), y[:6, h // 2].double()]) for x, y in zip(case.rows[0], (case.k, case.v)))
        score = torch.where(keep, case.q[:6, h].double() @ k.T, -math.inf)
        top2 = score.topk(2, 1).values
        clear = top2[:, 0] - top2[:, 1] > 2.0 ** -20 * (case.q[:6, h].double().abs() @ k.abs().T).amax(1) + 100
        best = v[score.argmax(1)]
        assert clear.any()
        assert torch.equal(out[:6, h][clear].double(), best[clear])


@pytest.mark.parametrize("scale_log2", [-64, -20, 0, 30, 64])
def test_value_scales_of_a_wide_range(q_, scale_log2):
    """New tokens of the size of the cache's values, whatever the scale."""
    case = Case(q_, [150], [10], 4, 2, 64, 16, F8, "tree", seed=44)
    case.vs.fill_(2.0 ** scale_log2)
    case.v.mul_(2.0 ** scale_log2)
    out, lse = case.run(0.1)
    case.check(0.1, out, lse)


@pytest.mark.parametrize("heads,dim", [(1, 128), (3, 64)])
def test_long_chain_with_values_that_are_not_finite(q_, heads, dim):
    """What is added back to the rows that see it is found in a time that no wait of the kernel takes for a fault."""
    n, at = 150000, [3, 70001, 149990]
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = _rows(n, heads, dim, g), _rows(n, 1, dim, g), _rows(n, 1, dim, g)
    cache = q_.kv_cache(*(torch.zeros((1, 1, 16, dim), dtype=BF, device="cuda") for _ in range(2)), _i32([[0]]))
    ws = q_.workspace(q_.qerl_tree_attention_workspace_size(n, heads, 1, dim, 1))

    def run():
        out, lse = torch.empty((n, heads, dim), dtype=BF, device="cuda"), torch.empty((n, heads), device="cuda")
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        q_.check(q_.qerl_tree_attention(cache, q, k, v, _i32([0, n]), _i32([5]), None, dim ** -0.5, out, lse, ws))
        end.record()
        assert q_.qerl_read_status(ws) == q_.QERL_OK
        return out, lse, start.elapsed_time(end)

    for x, a in enumerate(at):
        v[a, 0, 7 * x + 1] = (math.inf, math.nan, -math.inf)[x]
    out, lse, slow = run()
    for x, a in enumerate(at):
        v[a, 0, 7 * x + 1] = 0
    clean, lse2, fast = run()
    assert torch.equal(lse, lse2) and torch.isfinite(clean.float()).all()
    for x, a in enumerate(at):
        column = out[:, :, 7 * x + 1].float()
        assert (column[a:] == math.inf).all() if x == 0 else not torch.isfinite(column[a:]).any()
        assert torch.equal(out[:a, :, 7 * x + 1], clean[:a, :, 7 * x + 1])
        out[:, :, 7 * x + 1] = clean[:, :, 7 * x + 1]
    assert torch.equal(out, clean)
    assert slow < 20 * fast  # (one token after the other in every thread: 80 times)


@pytest.mark.parametrize("heads,hk", [(1, 1), (2, 2), (3, 1), (14, 2), (12, 1), (80, 1)])
@pytest.mark.parametrize("counts", [[700], [513, 1, 0, 400, 128]])
def test_chains_of_many_blocks(q_, heads, hk, counts):
    """In order, the segments of a sequence have different lengths on the line."""
    case = Case(q_, [150, 0, 20, 129, 1][:len(counts)], counts, heads, hk, 64, 16, BF, "chain", seed=heads)
    out, lse = case.run(0.125)
    case.check(0.125, out, lse)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,hk", [(6, 2), (9, 1)])
def test_parts_of_prompts_over_the_cache(q_, dtype, heads, hk):
    """Long chains behind rows in the cache: whole tiles of both, with and without a mask of their own."""
    case = Case(q_, [700, 129, 0], [520, 77, 260], heads, hk, 128, 32, dtype, "chain", seed=heads, pad=1)
    out, lse = case.run(0.09)
    case.check(0.09, out, lse)
    t = torch.arange(520, device="cuda")
    bits = torch.zeros((case.tokens, 9), dtype=torch.int64, device="cuda")  # the same as a mask
    for s in range(3):
        for w in range(9):
            n = case.counts[s]
            seen = (t[:n] + 1 - 64 * w).clamp(0, 64)
            bits[case.cu[s]:case.cu[s] + n, w] = torch.where(seen == 64, -1, (torch.ones_like(seen) << seen.clamp(max=63)) - 1)
    case.mask = bits
    out2, lse2 = case.run(0.09)
    case.check(0.09, out2, lse2)


@pytest.mark.parametrize("heads,hk,count", [(1024, 1, 2), (1024, 2, 1), (1023, 3, 3)])
def test_the_largest_groups(q_, heads, hk, count):
    case = Case(q_, [140], [count], heads, hk, 64, 16, BF, "tree", seed=heads)
    out, lse = case.run(0.125)
    case.check(0.125, out, lse)
