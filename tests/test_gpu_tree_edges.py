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


def check_mixed(case, scale, out, lse):
    group = case.heads // case.hk
    for s, (m, c) in enumerate(zip(case.lens, case.counts)):
        rows = slice(case.cu[s], case.cu[s] + c)
        if c == 0:
            continue
        keep = torch.cat([torch.ones((c, m), dtype=torch.bool, device="cuda"), case.keep[s]], 1)
        for h in range(case.heads):
            j = h // group
            k, v = (torch.cat([x[j].double() * f[j].double(), y[rows, j].double()])
                    for x, f, y in zip(case.rows[s], (case.ks, case.vs), (case.k, case.v)))
            o, l, to, tl = mixed64(case.q[rows, h], k, v, scale, keep, m)
            assert_within(out[rows, h], o, to, f"sequence {s} head {h}")
            none = torch.isinf(l)
            assert (lse[rows, h][none] == -math.inf).all() and (out[rows, h][none] == 0).all()
            assert_within(lse[rows, h][~none], l[~none], tl[~none], f"lse of sequence {s} head {h}")


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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("count", [1, 9])
def test_weights_of_a_cache_row_keep_the_bits_of_fp16(q_, dim, count):
    """Two rows with values 1 and -1: the output is the difference of two weights near 1/2.  The larger is exact;
    a rounding of the smaller to bf16 puts it off by up to 2^-10, twice what fp16 may."""
    n, hk = 300, 16
    case = Case(q_, [2] * n, [count] * n, hk, hk, dim, 2, F8, "any", seed=dim)
    case.mask.zero_()
    for keep in case.keep:
        keep.zero_()
    case.pages[1][:, :, 0], case.pages[1][:, :, 1] = 0x38, 0xB8  # 1 and -1
    case.vs.fill_(1.0)
    scale = 0.005
    out, lse = case.run(scale)
    # all sequences at once: [n, hk, 2, dim] keys
    k = torch.stack([x[0].double() for x in case.rows]) * case.ks.double()[:, None, None]
    q = case.q.view(n, count, hk, dim).double()
    s = torch.einsum("nchd,nhjd->nchj", q, k) * scale
    p = torch.softmax(s, -1)
    want = (p[..., 0] - p[..., 1])[..., None].expand(n, count, hk, dim)
    d = 2.0 ** -20 * (1.0 + scale * torch.einsum("nchd,nhjd->nchj", q.abs(), k.abs()).amax(-1))[..., None]
    assert want.abs().median() < 0.05
    assert_within(out.view(n, count, hk, dim), want, 2.0 ** -8 * want.abs() + 4 * d + 2.0 ** -11 + 2.0 ** -31)


@pytest.mark.parametrize("heads,hk,dim,page", [(40, 8, 128, 24), (45, 3, 64, 100), (28, 4, 128, 32)])
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
def test_e4m3_batches_at_the_bound_of_fp16(q_, heads, hk, dim, page, kind):
    case = Case(q_, [5, 0, 700, 128, 129, 3000, 0, 383, 64], [3, 7, 0, 33, 16, 50, 61, 1, 150], heads, hk, dim, page, F8,
                kind, seed=heads)
    out, lse = case.run(1 / math.sqrt(dim))
    check_mixed(case, 1 / math.sqrt(dim), out, lse)


def test_every_e4m3_key(q_):
    """One row per sequence and a query of one element per head: lse is the score, the key's value."""
    codes = [c for c in range(256) if c & 0x7F != 0x7F]
    case = Case(q_, [1] * 4, [1] * 4, 64, 1, 64, 4, F8, "any", seed=1)
    case.mask.zero_()
    case.ks.fill_(1.0)
    values = torch.tensor((codes + [0, 0])[:256], dtype=torch.uint8, device="cuda").view(4, 64)
    for s in range(4):
        case.pages[0][int(case.cache.tensors[2][s, 0]), 0, 0] = values[s]
    case.q.copy_(torch.eye(64, device="cuda").to(BF).expand(4, 64, 64))
    for scale in (1.0, 256.0):
        _, lse = case.run(scale)
        want = values.view(F8).double() * scale
        # one product of two exact factors: the factor of the score and lse's own steps
        assert_within(lse, want, 2.0 ** -20 * want.abs(), f"scale {scale}")


# ---- value scales ---------------------------------------------------------------


@pytest.mark.parametrize("scale", [-0.01, 0.0, -0.0, 2.0 ** -80, -2.0 ** -100, 2.0 ** 39, 2.0 ** 41, -2.0 ** 100])
@pytest.mark.parametrize("same_size", [False, True])
@pytest.mark.parametrize("count", [10, 70])
def test_value_scales_of_any_size_and_sign(q_, scale, same_size, count):
    """New tokens' values near 1, or as large as the cache's.  Some tokens see no new ones: theirs are the cache's
    values alone, however small those are beside the new tokens'."""
    case = Case(q_, [150, 700], [count, 12], 8, 2, 64, 16, F8, "any", seed=44)
    case.vs.fill_(scale)
    if same_size:
        case.v.mul_(abs(scale))
    case.mask[::5] = 0
    for s, keep in enumerate(case.keep):
        rows = torch.arange(case.cu[s], case.cu[s + 1], device="cuda")
        keep[rows % 5 == 0] = False
    out, lse = case.run(0.1)
    group = case.heads // case.hk
    for s, (m, c) in enumerate(zip(case.lens, case.counts)):
        rows = slice(case.cu[s], case.cu[s] + c)
        keep = torch.cat([torch.ones((c, m), dtype=torch.bool, device="cuda"), case.keep[s]], 1)
        for h in range(case.heads):
            j = h // group
            k = torch.cat([case.rows[s][0][j].double() * case.ks[j].double(), case.k[rows, j].double()])
            # in units of 2^-100 of the values, so that the bound's 1e-30 is small
            v = torch.cat([case.rows[s][1][j].double() * scale, case.v[rows, j].double()]) * 2.0 ** 100
            o, l, to, tl = mixed64(case.q[rows, h], k, v, 0.1, keep, m)
            assert_within(out[rows, h].double() * 2.0 ** 100, o, to, f"sequence {s} head {h}")
            assert_within(lse[rows, h], l, tl)


def test_value_scales_differ_by_head_and_over_many_ctas(q_):
    """A long sequence whose segments are joined, with a scale of either side of 1 for its heads."""
    case = Case(q_, [20011], [30], 8, 4, 128, 32, F8, "tree", seed=45)
    case.vs.copy_(torch.tensor([-3.0, 2.0 ** -70, 2.0 ** 70, 0.02]))
    out, lse = case.run(0.09)
    group = 2
    keep = torch.cat([torch.ones((30, 20011), dtype=torch.bool, device="cuda"), case.keep[0]], 1)
    for h in range(8):
        j = h // group
        k = torch.cat([case.rows[0][0][j].double() * case.ks[j].double(), case.k[:, j].double()])
        v = torch.cat([case.rows[0][1][j].double() * case.vs[j].double(), case.v[:, j].double()])
        o, l, to, tl = mixed64(case.q[:, h], k, v, 0.09, keep, 20011)
        assert_within(out[:, h], o, to, f"head {h}")
        assert_within(lse[:, h], l, tl)


def test_key_scales_of_any_size_and_sign(q_):
    """0 makes the cache's scores 0; one that is not finite reaches the outputs of its heads."""
    for scale in (0.0, -0.0, -0.01, 2.0 ** -120, math.nan, math.inf):
        case = Case(q_, [150, 700], [10, 70], 8, 2, 64, 16, F8, "any", seed=46)
        case.ks[1] = scale
        out, lse = case.run(0.1)
        if math.isfinite(scale):
            check_mixed(case, 0.1, out, lse)
        else:
            assert not torch.isfinite(out[:, 4:].float()).any() and not torch.isfinite(lse[:, 4:]).any()
            assert torch.isfinite(out[:, :4].float()).all() and torch.isfinite(lse[:, :4]).all()


# ---- rows do not see what they do not attend to -----------------------------------


# Many sequences, so that a CTA's stretch holds several key tiles: groups of new tokens of up to 128 rows (whose
# two query tiles share them) and of more.
LONG = [(24, 1500, 20, 16, 4), (12, 2100, 70, 8, 4), (20, 1300, 300, 4, 2)]


def _long(q_, seqs, rows, count, heads, hk, dtype, dim, seed):
    r = random.Random(seed)
    return Case(q_, [rows + r.randint(-300, 300) for _ in range(seqs)], [count - r.randint(0, 3) for _ in range(seqs)],
                heads, hk, dim, 32, dtype, "any", seed=seed)


@pytest.mark.parametrize("seqs,rows,count,heads,hk", LONG)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_a_large_key_changes_no_bit_of_rows_that_do_not_see_it(q_, seqs, rows, count, heads, hk, dim, dtype):
    """Its score moves the reference of the rows that do, far above the cache's scores before it."""
    case = _long(q_, seqs, rows, count, heads, hk, dtype, dim, seed=61)
    clean, lse = case.run(0.1)
    hit = torch.zeros(case.tokens, dtype=torch.bool, device="cuda")
    for s in range(seqs):
        for at in (1, case.counts[s] - 2):
            case.k[case.cu[s] + at] *= 64
            hit[case.cu[s]:case.cu[s + 1]] |= case.keep[s][:, at]
    assert hit.any() and not hit.all()
    out, lse2 = case.run(0.1)
    assert (out[hit] != clean[hit]).any()
    assert torch.equal(lse[~hit], lse2[~hit])
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("seqs,rows,count,heads,hk", LONG)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_masked_drafts_hold_anything_in_items_of_many_tiles(q_, seqs, rows, count, heads, hk, dim, dtype):
    """A value or key that is not finite reaches the tokens that see it and no others, where a tile with masks is
    not the first of its item, the reference has moved, and the two query tiles exchange their outputs."""
    case = _long(q_, seqs, rows, count, heads, hk, dtype, dim, seed=62)
    clean, lse = case.run(0.1)
    check = check_mixed if dtype == F8 else lambda c, *a: c.check(*a)
    check(case, 0.1, clean, lse)
    kinds = [math.nan, math.inf, -math.inf]
    places = [[0, 3, case.counts[s] - 1] for s in range(seqs)]
    for s in range(seqs):  # values: columns 7, 8, 9 of the tokens that see them
        for x, at in enumerate(places[s]):
            case.v[case.cu[s] + at, :, 7 + x] = kinds[(s + x) % 3]
    out, lse2 = case.run(0.1)
    assert torch.equal(lse, lse2)
    for s in range(seqs):
        mine = slice(case.cu[s], case.cu[s + 1])
        for x, at in enumerate(places[s]):
            reached = case.keep[s][:, at]
            column = out[mine, :, 7 + x]
            assert not torch.isfinite(column[reached].float()).any()
            assert torch.equal(column[~reached], clean[mine, :, 7 + x][~reached])
    rest = [c for c in range(dim) if c not in (7, 8, 9)]
    assert torch.equal(out[:, :, rest], clean[:, :, rest])
    hit = torch.zeros(case.tokens, dtype=torch.bool, device="cuda")
    for s in range(seqs):
        for x, at in enumerate(places[s]):
            case.k[case.cu[s] + at, :, 5] = kinds[(s + x) % 3]
            hit[case.cu[s]:case.cu[s + 1]] |= case.keep[s][:, at]
    out, lse2 = case.run(0.1)
    assert hit.any() and not hit.all()
    assert torch.equal(lse[~hit], lse2[~hit]) and torch.equal(out[~hit], clean[~hit])


# ---- numbers of sequences -----------------------------------------------------


# Up to 32 are looked through by one warp, up to the threads (512; E4M3 640) in one round, more in several.
@pytest.mark.parametrize("n", [32, 33, 96, 512, 513, 640, 641, 1300])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_numbers_of_sequences_and_offsets_that_break_the_rules(q_, n, dtype):
    r = random.Random(n)
    lens = [r.choice([0, 3, 40, 129]) for _ in range(n)]
    counts = [r.choice([0, 1, 2, 5]) for _ in range(n)]
    for i in (0, 1, -1):
        counts[i] = 0
    counts[2] = counts[n // 2] = counts[-2] = 3
    lens[n // 3], counts[n // 3] = 5000, 7
    case = Case(q_, lens, counts, 4, 2, 64, 16, dtype, "tree", seed=n, lead=2, tail=3)
    out, lse = case.run(0.125)
    (check_mixed if dtype == F8 else lambda c, *a: c.check(*a))(case, 0.125, out, lse)
    for x in (out, lse):
        assert (x[:2] == 5).all() and (x[-3:] == 5).all()
    good = case.cu
    for at, to in ((0, -1), (2, good[3] + 1), (n // 2, good[n // 2 + 1] + 1), (n - 2, good[n - 1] + 2),
                   (n - 1, good[n - 2] - 1), (n, case.tokens + 1)):
        case.cu = list(good)
        case.cu[at] = to
        broken, lse2 = case.run(0.125, status="QERL_ERR_RANGE")
        assert (broken == 5).all() and (lse2 == 5).all(), f"offset {at}"
    case.cu = good
    again, lse2 = case.run(0.125)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# ---- the largest calls ---------------------------------------------------------


def _chain(q_, n, g):
    q, k, v = (torch.randn((n, 1, 64), generator=g, device="cuda").to(BF) for _ in range(3))
    cache = q_.kv_cache(*(torch.zeros((1, 1, 16, 64), dtype=BF, device="cuda") for _ in range(2)), _i32([[0]]))
    out, lse = torch.full((n, 1, 64), 5.0, dtype=BF, device="cuda"), torch.full((n, 1), 5.0, device="cuda")
    ws = q_.workspace(q_.qerl_tree_attention_workspace_size(n, 1, 1, 64, 1))
    q_.check(q_.qerl_tree_attention(cache, q, k, v, _i32([0, n]), _i32([0]), None, 0.125, out, lse, ws))
    return q, k, v, out, lse, q_.STATUS_NAMES[q_.qerl_read_status(ws)]


def test_the_longest_chain_and_one_token_more(q_):
    g = torch.Generator(device="cuda").manual_seed(71)
    n = 2 ** 20
    q, k, v, out, lse, status = _chain(q_, n, g)
    assert status == "QERL_OK"
    at = torch.tensor([0, 1, 255, 256, 2 ** 19 + 3, n - 129, n - 1], device="cuda")
    keep = torch.arange(n, device="cuda") <= at[:, None]
    o, l, to, tl = masked64(q[at, 0], k[:, 0], v[:, 0], 0.125, keep, "bf16")
    assert_within(out[at, 0], o, to)
    assert_within(lse[at, 0], l, tl)
    _, _, _, out, lse, status = _chain(q_, n + 1, g)
    assert status == "QERL_ERR_RANGE"
    assert (out == 5).all() and (lse == 5).all()


@pytest.mark.parametrize("dtype", [BF, F8])
def test_the_widest_masks(q_, dtype):
    case = Case(q_, [100, 300], [9, 4], 4, 2, 64, 16, dtype, "any", seed=72, words=2 ** 14)
    out, lse = case.run(0.125)
    (check_mixed if dtype == F8 else lambda c, *a: c.check(*a))(case, 0.125, out, lse)
