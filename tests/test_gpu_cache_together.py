"""The operators of the cache as a rollout uses them: packed prompts within a window, forked into groups, drafts
verified and appended, single tokens within the window, ended sequences' pages given back."""
import random

import pytest
import torch

from attention_reference import assert_within
from masked_reference import masked64, window_keep

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HEADS, HK, DIM, PAGE, WINDOW, SINKS, SCALE = 8, 2, 64, 16, 40, 4, 0.125


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Rollout:
    """A pool, its table, and what every sequence holds: rows of k and v [tokens, kv_heads, dim] as the cache has
    them (fp64)."""

    def __init__(self, q_, dtype, seqs, pool=150, seed=0):
        self.q_, self.dtype = q_, dtype
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.r = random.Random(seed)
        shape = (pool, HK, PAGE, DIM)
        self.pages = [torch.zeros(shape, dtype=BF, device="cuda").to(dtype) for _ in range(2)]
        self.scale = None if dtype == BF else torch.full((HK,), 1 / 64, device="cuda")
        self.table = torch.full((seqs, 16), -1, dtype=torch.int32, device="cuda")
        self.free = self.r.sample(range(pool), pool)
        self.held = [[torch.zeros((0, HK, DIM), dtype=torch.float64, device="cuda")] * 2 for _ in range(seqs)]
        self.freq = 1e4 ** (-torch.arange(DIM // 2, dtype=torch.float64, device="cuda") / (DIM // 2))
        self.describe()

    def describe(self):
        self.cache = self.q_.kv_cache(*self.pages, self.table, self.scale, self.scale)

    def rows(self, n, heads):
        return torch.randn((n, heads, DIM), generator=self.g, device="cuda").to(BF)

    def length(self, s):
        return self.held[s][0].shape[0]

    def grow(self, s, tokens):
        """Pages for that many tokens more."""
        for j in range(-(-self.length(s) // PAGE), -(-(self.length(s) + tokens) // PAGE)):
            self.table[s, j] = self.free.pop()

    def kept(self, s, p):
        """A row of k and of v as the cache holds it (how it comes there is the append's own test)."""
        got = []
        for x in self.pages:
            x = x.view(torch.uint8 if self.dtype == F8 else BF)[int(self.table[s, p // PAGE]), :, p % PAGE].view(self.dtype)
            got.append(x.double()[None] * (1.0 if self.scale is None else self.scale[0].double()))
        return got

    def append(self, q, k, v, places, seqs, rotate=True, take=None):
        """k and v at places of sequences (those of `take`, if given): (rotated q, rotated k)."""
        take = torch.ones(len(places), dtype=torch.bool) if take is None else take
        ws = self.q_.workspace(self.q_.qerl_rope_append_workspace_size())
        where = _i32([p if t else -1 for p, t in zip(places, take)])
        freq = self.freq if rotate else self.freq[:0]
        qr, kr = self.q_.rope_append(self.cache, q, k, v, where, freq, seq_ids=_i32(seqs), ws=ws)
        assert self.q_.qerl_read_status(ws) == 0
        for i, (s, t) in enumerate(zip(seqs, take)):
            if t:
                assert places[i] == self.length(s)
                self.held[s] = [torch.cat(x) for x in zip(self.held[s], self.kept(s, places[i]))]
        return qr, kr

    def near(self, got, q, k, v, keep, weights, what):
        out, lse = got
        for h in range(HEADS):
            o, l, to, tl = masked64(q[:, h], k[:, h // 4], v[:, h // 4], SCALE, keep, weights)
            assert_within(out[:, h], o, to, f"{what} head {h}")
            assert_within(lse[:, h], l, tl, f"{what} lse of head {h}")

    def decode(self, seqs):
        """One new token of every sequence of `seqs` (length 0 for the others), appended and attended from."""
        n = self.table.shape[0]
        for s in seqs:
            self.grow(s, 1)
        q, k, v = self.rows(n, HEADS), self.rows(n, HK), self.rows(n, HK)
        take = [s in seqs for s in range(n)]
        qr, _ = self.append(q, k, v, [self.length(s) for s in range(n)], list(range(n)), take=take)
        qr[[s for s in range(n) if s not in seqs]] = 0
        return qr, self.attend(qr, seqs)

    def attend(self, qr, seqs):
        n = self.table.shape[0]
        lengths = _i32([self.length(s) if s in seqs else 0 for s in range(n)])
        ws = self.q_.workspace(self.q_.qerl_decode_attention_workspace_size(n, HEADS, HK, DIM))
        out, lse = self.q_.window_decode_attention(self.cache, qr, lengths, WINDOW, SINKS, SCALE, ws)
        assert self.q_.qerl_read_status(ws) == 0
        weights = "split" if self.dtype == BF else "fp16"
        for s in seqs:
            at = torch.arange(self.length(s), device="cuda")
            self.near((out[s:s + 1], lse[s:s + 1]), qr[s:s + 1], *self.held[s], window_keep(at[-1:], at, WINDOW, SINKS),
                      weights, f"token of sequence {s}")
        return out, lse


@pytest.mark.parametrize("dtype", [BF, F8])
def test_a_rollout(q_, dtype):
    prompts, group = [70, 33, 128], 2
    roll = Rollout(q_, dtype, len(prompts) * (1 + group))
    # prompts
    seqs = [s for s, m in enumerate(prompts) for _ in range(m)]
    places = [p for m in prompts for p in range(m)]
    for s, m in enumerate(prompts):
        roll.grow(s, m)
    q, k, v = roll.rows(len(seqs), HEADS), roll.rows(len(seqs), HK), roll.rows(len(seqs), HK)
    qr, kr = roll.append(q, k, v, places, seqs)
    cu = [0, 70, 103, 231]
    out, lse = q_.window_prompt_attention(qr, kr, v, _i32(cu), WINDOW, SINKS, SCALE)
    for a, b in zip(cu, cu[1:]):
        at = torch.arange(b - a, device="cuda")
        roll.near((out[a:b], lse[a:b]), qr[a:b], kr[a:b], v[a:b], window_keep(at, at, WINDOW, SINKS), "bf16", "prompt")
    # groups of rollouts
    parents = [s for s in range(3) for _ in range(group)]
    children = list(range(3, 9))
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.kv_fork(roll.cache, _i32(parents), _i32(children), _i32([prompts[s] for s in parents]),
               _i32([roll.free.pop() for _ in children]), ws)
    assert q_.qerl_read_status(ws) == 0
    for s, c in zip(parents, children):
        roll.held[c] = list(roll.held[s])
    roll.decode(children)
    # drafts: verified, and one branch of each appended
    for _ in range(3):
        count = 6
        n = len(children) * count
        q, k, v = roll.rows(n, HEADS), roll.rows(n, HK), roll.rows(n, HK)
        seen = []
        for _ in children:
            for t in range(count):
                parent = roll.r.randint(-1, t - 1)
                seen.append((seen[parent - t] if parent >= 0 else 0) | 1 << t)
        depth = torch.tensor([bin(x).count("1") - 1 for x in seen])
        start = torch.tensor([roll.length(c) for c in children]).repeat_interleave(count)
        qr, kr = q_.rope_append(None, q, k, None, (start + depth).to(torch.int32).cuda(), roll.freq)
        lengths = [0] * 3 + [roll.length(c) for c in children]  # the prompts have no new tokens now
        offsets = [0, 0, 0] + [count * i for i in range(len(children) + 1)]
        ws = q_.workspace(q_.qerl_tree_attention_workspace_size(n, HEADS, HK, DIM, 9))
        out, lse = q_.tree_attention(roll.cache, qr, kr, v, _i32(offsets), _i32(lengths),
                                     torch.tensor(seen, dtype=torch.int64, device="cuda")[:, None], SCALE, ws)
        assert q_.qerl_read_status(ws) == 0
        for i, c in enumerate(children):
            rows = slice(i * count, (i + 1) * count)
            keep = torch.tensor([[bool(x >> j & 1) for j in range(count)] for x in seen[rows]], device="cuda")
            keep = torch.cat([torch.ones((count, roll.length(c)), dtype=torch.bool, device="cuda"), keep], 1)
            keys, values = (torch.cat([h, x[rows].double()]) for h, x in zip(roll.held[c], (kr, v)))
            roll.near((out[rows], lse[rows]), qr[rows], keys, values, keep, "bf16", f"draft of {c}")
        # a branch of each child's
        accepted = []
        for i in range(len(children)):
            leaf = seen[i * count + roll.r.randrange(count)]
            accepted += [bool(leaf >> t & 1) for t in range(count)]
        for i, c in enumerate(children):
            roll.grow(c, sum(accepted[i * count:(i + 1) * count]))
        roll.append(None, kr, v, (start + depth).tolist(), [c for c in children for _ in range(count)], rotate=False,
                    take=accepted)
    qr, before = roll.decode(children)
    # the prompts and two answers end: their pages and those behind the others' windows are given up
    live = children[2:]
    for s in live:
        for j in range(-(-SINKS // PAGE), (roll.length(s) - WINDOW) // PAGE):
            roll.table[s, j] = -1
    lengths = _i32([roll.length(s) if s in live else 0 for s in range(9)])
    ws = q_.workspace(q_.qerl_kv_compact_workspace_size(roll.pages[0].shape[0]))
    used = {int(x) for s in live for x in roll.table[s, :-(-roll.length(s) // PAGE)].tolist() if x >= 0}
    table, count = q_.kv_compact(roll.cache, lengths, ws)
    assert q_.qerl_read_status(ws) == 0
    assert count.item() == len(used)
    assert {int(x) for s in live for x in table[s, :-(-roll.length(s) // PAGE)].tolist() if x >= 0} == set(range(len(used)))
    for x in roll.pages:  # the tail of the pool is somebody else's now
        x[len(used):] = float("nan")
    roll.table = table.contiguous()
    roll.describe()
    after = roll.attend(qr, live)
    for a, b in zip(before, after):
        assert torch.equal(a[live], b[live])
    roll.free = list(range(len(used), roll.pages[0].shape[0]))
    roll.decode(live)
