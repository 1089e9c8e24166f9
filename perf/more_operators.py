"""What the operators around the paged cache that go beyond one token and one prompt are measured on.

  tree     attention of drafted tokens (a tree or a chain per sequence) over the paged cache
  wdecode  attention of one new token per sequence over a window of the cache and its first rows (sinks)
  wprompt  causal attention of packed prompts within a window, with sinks
  fork     children of a sequence: its full pages shared, the rows of its last page copied
  compact  the pages in use moved to the front of the pool

`own` False computes each in its plain form (elementary torch operations, 32-bit arithmetic, one
rounding at the end); `own` True calls the library's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

#: (query heads, key-value heads, head size) of the decoder blocks the cases stand for.
_BLOCKS = [(16, 2, 128), (28, 4, 128), (40, 8, 128), (32, 8, 64), (8, 8, 64), (12, 1, 128), (45, 3, 64), (10, 2, 64)]
_PAGES = [1, 8, 16, 24, 32, 64, 100, 128]


def listed():
    return [
        # One request whose next tokens were drafted as a chain: latency.
        {"name": "tree-chain-one", "op": "tree", "heads": 28, "kv_heads": 4, "dim": 128, "cache": "bf16", "page": 16,
         "seqs": 1, "max_len": 777, "ragged": False, "nodes": 5, "chain": True},
        # A batch of rollouts at different lengths, a small tree each.
        {"name": "tree-ragged", "op": "tree", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64,
         "seqs": 48, "max_len": 8192, "ragged": True, "nodes": 25, "chain": False},
        # Large trees over an 8-bit cache: as much arithmetic as traffic.
        {"name": "tree-batch-e4m3", "op": "tree", "heads": 28, "kv_heads": 4, "dim": 128, "cache": "e4m3", "page": 32,
         "seqs": 64, "max_len": 6000, "ragged": False, "nodes": 61, "chain": False},
        # Small heads, many short rollouts.
        {"name": "tree-small-heads", "op": "tree", "heads": 32, "kv_heads": 8, "dim": 64, "cache": "bf16", "page": 24,
         "seqs": 96, "max_len": 2500, "ragged": True, "nodes": 30, "chain": False},
        # One long chat that keeps a window: latency.
        {"name": "wdecode-one", "op": "wdecode", "heads": 16, "kv_heads": 2, "dim": 128, "cache": "bf16", "page": 16,
         "seqs": 1, "max_len": 50001, "ragged": False, "window": 1000, "sinks": 4},
        # A batch of rollouts, most of them past the window.
        {"name": "wdecode-batch", "op": "wdecode", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64,
         "seqs": 192, "max_len": 12000, "ragged": True, "window": 4096, "sinks": 64},
        # A batch of prompts of different lengths, packed.
        {"name": "wprompt-packed", "op": "wprompt", "heads": 28, "kv_heads": 4, "dim": 128, "seqs": 10, "max_len": 3001,
         "ragged": True, "window": 500, "sinks": 4},
        # One long prompt.
        {"name": "wprompt-long", "op": "wprompt", "heads": 40, "kv_heads": 8, "dim": 128, "seqs": 1, "max_len": 16384,
         "ragged": False, "window": 2048, "sinks": 16},
        # A few answers to one prompt: latency.
        {"name": "fork-one", "op": "fork", "heads": 16, "kv_heads": 2, "dim": 128, "cache": "bf16", "page": 16, "seqs": 1,
         "max_len": 777, "ragged": False, "children": 7},
        # Groups of rollouts of a batch of prompts.
        {"name": "fork-groups", "op": "fork", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64,
         "seqs": 48, "max_len": 4000, "ragged": True, "children": 8},
        # A small pool after a few sequences ended: latency.
        {"name": "compact-small", "op": "compact", "heads": 16, "kv_heads": 2, "dim": 128, "cache": "bf16", "page": 16,
         "seqs": 6, "max_len": 300, "ragged": True, "spare": 0.5, "group": 1},
        # A large pool whose tail is wanted for something else.
        {"name": "compact-pool", "op": "compact", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64,
         "seqs": 96, "max_len": 8192, "ragged": True, "spare": 1.0, "group": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "wdecode", "wprompt", "fork", "compact"])
    heads, kv_heads, dim = rng.choice(_BLOCKS)
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "ragged": rng.random() < 0.6}
    if op != "wprompt":
        case |= {"cache": rng.choice(["bf16", "e4m3"]), "page": rng.choice(_PAGES)}
    if op == "tree":
        nodes = _log_int(rng, 1, 200)
        case |= {"seqs": _log_int(rng, 1, 128), "max_len": _log_int(rng, 1, 60000), "nodes": nodes,
                 "chain": rng.random() < 0.3}
    elif op == "wdecode":
        case |= {"seqs": _log_int(rng, 1, 256), "max_len": _log_int(rng, 1, 60000), "window": _log_int(rng, 1, 8192),
                 "sinks": rng.choice([0, 1, 4, 16, 64, 129])}
    elif op == "wprompt":
        case |= {"seqs": _log_int(rng, 1, 16), "max_len": _log_int(rng, 1, 12000), "window": _log_int(rng, 1, 4096),
                 "sinks": rng.choice([0, 1, 4, 16, 64, 129, 300])}
    elif op == "fork":
        case |= {"page": max(case["page"], 8), "seqs": _log_int(rng, 1, 64), "max_len": _log_int(rng, 1, 4000),
                 "children": rng.randint(1, 16)}
    else:
        case |= {"page": max(case["page"], 8), "seqs": _log_int(rng, 1, 128), "max_len": _log_int(rng, 1, 8000),
                 "spare": rng.uniform(0.1, 1.5), "group": rng.choice([1, 1, 2, 4, 8])}
    most = [work(c) for c in listed() if c["op"] == op]
    while any(work(case)[x] > max(w[x] for w in most) for x in ("bytes", "flops")):  # no dearer than the listed ones
        longer = "max_len" if case["max_len"] >= 2 * case["seqs"] else "seqs"
        case[longer] = (case[longer] * 2 + 1) // 3
    return case


def _lengths(case):
    """The sequences' lengths: the longest somewhere, the others spread over the logarithm of the range."""
    n, longest = case["seqs"], case["max_len"]
    if not case["ragged"]:
        return [longest] * n
    r = random.Random("%d %d" % (n, longest))
    lens = [_log_int(r, max(1, longest // 16), longest) for _ in range(n)]
    lens[r.randrange(n)] = longest
    return lens


def _nodes(case):
    """The drafted tokens of every sequence."""
    n, most = case["seqs"], case["nodes"]
    r = random.Random("%d %d nodes" % (n, most))
    return [r.randint((most + 1) // 2, most) for _ in range(n - 1)] + [most] if case["ragged"] else [most] * n


def _layout(case):
    """Of a pool to compact: every sequence's (first own page's place, shared pages, pages), the pages in
    use, the pool's pages and how many of those in use lie past the used ones' count."""
    page, group = case["page"], case["group"]
    rows, used = [], 0
    for i, m in enumerate(_lengths(case)):
        pages = -(-m // page)
        lead = rows[i - i % group] if i % group else None  # the group's first sequence: its prompt is shared
        shared = min(pages, lead[2] // 2) if lead else 0
        rows.append((used, shared, pages))
        used += pages - shared
    total = used + int(used * case["spare"])
    return rows, used, total, min(int(used * (1 - used / total)), total - used)


def _normal(shape, g, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _pages(case, total, g):
    """Key and value pages of the cache and the scales of an 8-bit one."""
    s = {}
    for name in ("k", "v"):
        pages = torch.empty((total, case["kv_heads"], case["page"], case["dim"]), device="cuda", dtype=torch.bfloat16)
        pages.normal_(generator=g)
        s[name + "_scale"] = None
        if case["cache"] == "e4m3":  # such a cache holds value / scale, with the scales set from the values' largest
            s[name + "_scale"] = torch.rand(case["kv_heads"], generator=g, device="cuda") * 0.01 + 0.008
            pages = (pages.float() / s[name + "_scale"][:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name + "_pages"] = pages
    return s


def _order(n, g):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32).cpu().numpy()


def _cache(case, lens, g, spare=0, rows=0):
    """Pages and the page table of sequences of these lengths (pages in no order, unused entries 0), with
    `spare` pages and `rows` table rows more."""
    used = [-(-m // case["page"]) for m in lens]
    order = _order(sum(used) + spare, g)
    table = np.zeros((len(lens) + rows, max(used)), dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(used)])
    for i, n in enumerate(used):
        table[i, :n] = order[at[i]:at[i] + n]
    s = _pages(case, sum(used) + spare, g)
    s |= {"table": torch.from_numpy(table).cuda(), "spare_pages": torch.from_numpy(order[at[-1]:].copy()).cuda()}
    return s


def _tree_mask(case, counts, g):
    """A random tree per sequence: bit j of a node's words is set for itself and its ancestors."""
    r = random.Random(int(torch.randint(1 << 30, (1,), generator=g, device="cuda").item()))
    words = -(-case["nodes"] // 64)
    mask = []
    for n in counts:
        seen = []
        for i in range(n):
            parent = r.randint(max(-1, i - 8), i - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        mask += seen
    flat = [(m >> (64 * w)) & (1 << 64) - 1 for m in mask for w in range(words)]
    return torch.from_numpy(np.array(flat, dtype=np.uint64).view(np.int64).reshape(-1, words)).cuda()


def _offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    h, hk, d, op = case["heads"], case["kv_heads"], case["dim"], case["op"]
    lens = _lengths(case)
    n = len(lens)
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if op == "tree":
        s |= _cache(case, lens, g)
        counts = _nodes(case)
        tokens = sum(counts)
        s["q"], s["k"], s["v"] = _normal((tokens, h, d), g, 1.5), _normal((tokens, hk, d), g), _normal((tokens, hk, d), g)
        s["cu"], s["lengths"] = _offsets(counts), torch.tensor(lens, dtype=torch.int32).cuda()
        s["mask"] = None if case["chain"] else _tree_mask(case, counts, g)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((tokens, h), device="cuda")
    elif op == "wdecode":
        s |= _cache(case, lens, g)
        s["q"], s["lengths"] = _normal((n, h, d), g, 1.5), torch.tensor(lens, dtype=torch.int32).cuda()
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((n, h), device="cuda")
    elif op == "wprompt":
        tokens = sum(lens)
        s["q"], s["k"], s["v"] = _normal((tokens, h, d), g, 1.5), _normal((tokens, hk, d), g), _normal((tokens, hk, d), g)
        s["cu"] = _offsets(lens)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((tokens, h), device="cuda")
    elif op == "fork":
        kids = n * case["children"]
        s |= _cache(case, lens, g, spare=kids, rows=kids)
        s["parents"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(case["children"])
        s["children"] = torch.arange(n, n + kids, dtype=torch.int32, device="cuda")
        s["lengths"] = torch.tensor(lens, dtype=torch.int32).cuda().repeat_interleave(case["children"])
        s["new_pages"] = s["spare_pages"]
    else:
        rows, used, total, moves = _layout(case)
        low, high = _order(used, g)[:used - moves], _order(total - used, g)[:moves] + used
        at = np.concatenate([low, high])[_order(used, g)]
        table = np.zeros((n, max(r[2] for r in rows)), dtype=np.int32)
        for i, (first, shared, pages) in enumerate(rows):
            table[i, :shared] = table[i - i % case["group"], :shared]
            table[i, shared:pages] = at[first:first + pages - shared]
        s |= _pages(case, total, g)
        s["table"], s["lengths"] = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        s["new_table"], s["live"] = torch.empty_like(s["table"]), torch.empty(1, dtype=torch.int32, device="cuda")
    if own:  # the cache's descriptor and the workspace, made once and kept
        import nvfp4_weight_quantized_03_gb300 as q
        if "k_pages" in s:
            s["cache"] = q.kv_cache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"])
        s["ws"] = q.workspace({
            "tree": lambda: q.qerl_tree_attention_workspace_size(s["q"].shape[0], h, hk, d, n),
            "wdecode": lambda: q.qerl_decode_attention_workspace_size(n, h, hk, d),
            "wprompt": lambda: q.qerl_prompt_attention_workspace_size(s["q"].shape[0], h, hk, d, n),
            "fork": q.qerl_kv_fork_workspace_size,
            "compact": lambda: q.qerl_kv_compact_workspace_size(s["k_pages"].shape[0]),
        }[op]())
    return s


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- the library's calls ----------------------------------------------------


def _tree_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_tree_attention(s["cache"], s["q"], s["k"], s["v"], s["cu"], s["lengths"], s["mask"], s["scale"],
                                  s["out"], s["lse"], s["ws"]))
    return {"out": s["out"], "lse": s["lse"]}


def _wdecode_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_window_decode_attention(s["cache"], s["q"], s["lengths"], s["case"]["window"], s["case"]["sinks"],
                                           s["scale"], s["out"], s["lse"], s["ws"]))
    return {"out": s["out"], "lse": s["lse"]}


def _wprompt_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_window_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["case"]["window"], s["case"]["sinks"],
                                           s["scale"], s["out"], s["lse"], s["ws"]))
    return {"out": s["out"], "lse": s["lse"]}


def _fork_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_kv_fork(s["cache"], s["parents"], s["children"], s["lengths"], s["new_pages"], s["ws"]))
    return {"table": s["table"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _compact_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_kv_compact(s["cache"], s["lengths"], s["new_table"], s["live"], s["ws"]))
    return {"table": s["new_table"], "live": s["live"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


_OWN = {"tree": _tree_own, "wdecode": _wdecode_own, "wprompt": _wprompt_own, "fork": _fork_own, "compact": _compact_own}


# ---- the plain forms --------------------------------------------------------


def _bits(pages):
    """8-bit pages as bytes, which torch can index."""
    return pages if pages.dtype == torch.bfloat16 else pages.view(torch.uint8)


def _gathered(pages, table, scale):
    """[seqs, kv_heads, positions, dim] in fp32, in the order of the sequences' positions."""
    x = _bits(pages)[table.long()].view(pages.dtype).float().permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _softmax_product(scores, v):
    """(softmax(scores) v, log sum exp): scores [..., rows, positions] with -inf where masked."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total, (total.log() + top)[..., 0]


def _tree_plain(s):
    t, h, d = s["q"].shape
    k, v = _gathered(s["k_pages"], s["table"], s["k_scale"]), _gathered(s["v_pages"], s["table"], s["v_scale"])
    n, hk, longest, _ = k.shape
    most = s["case"]["nodes"]
    # the packed tokens laid out as [sequences, most], then back
    cu = s["cu"].long()
    row = torch.arange(t, device="cuda")
    seq = torch.bucketize(row, cu[1:], right=True)
    own_place = row - cu[seq]
    at = seq * most + own_place

    def padded(x):
        full = torch.zeros((n * most,) + x.shape[1:], device="cuda", dtype=x.dtype)
        full[at] = x
        return full.view((n, most) + x.shape[1:])

    new_k, new_v = (padded(s[x].float()).transpose(1, 2) for x in "kv")  # [n, kv_heads, most, d]
    q = padded(s["q"].float()).view(n, most, hk, h // hk, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    node = torch.arange(most, device="cuda")
    if s["mask"] is None:
        seen = padded((node <= own_place[:, None]).to(torch.uint8)).bool()
    else:
        seen = padded((s["mask"][:, node // 64] >> (node % 64) & 1).to(torch.uint8)).bool()  # [n, most, most]
    past = torch.arange(longest, device="cuda") >= s["lengths"][:, None]
    hidden = torch.cat([past[:, None, :].expand(n, most, longest), ~seen], -1)[:, None].repeat(1, 1, h // hk, 1)
    scores = (q @ torch.cat([k, new_k], 2).transpose(-1, -2)) * s["scale"]
    out, lse = _softmax_product(scores.masked_fill_(hidden, -math.inf), torch.cat([v, new_v], 2))
    out = out.view(n, hk, h // hk, most, d).permute(0, 3, 1, 2, 4).reshape(n * most, h, d)[at]
    return {"out": out.to(torch.bfloat16), "lse": lse.view(n, h, most).transpose(1, 2).reshape(n * most, h)[at]}


def _wdecode_plain(s):
    n, h, d = s["q"].shape
    window, sinks, page = s["case"]["window"], s["case"]["sinks"], s["case"]["page"]
    # the rows that any sequence can see: the first `sinks`, then the last `window`
    place = torch.arange(min(window + sinks, s["table"].shape[1] * page), device="cuda")
    skip = (s["lengths"].long() - window - sinks).clamp(min=0)[:, None]
    row = torch.where(place < sinks, place, place + skip).clamp(max=s["table"].shape[1] * page - 1)
    past = place + skip >= s["lengths"][:, None]
    number = torch.gather(s["table"].long(), 1, row // page)

    def rows(pages, scale):
        x = _bits(pages)[number, :, row % page].view(pages.dtype).float().transpose(1, 2)
        return x if scale is None else x * scale[None, :, None, None]

    k, v = rows(s["k_pages"], s["k_scale"]), rows(s["v_pages"], s["v_scale"])
    hk = k.shape[1]
    scores = (s["q"].float().view(n, hk, h // hk, d) @ k.transpose(-1, -2)) * s["scale"]
    out, lse = _softmax_product(scores.masked_fill(past[:, None, None, :], -math.inf), v)
    return {"out": out.reshape(n, h, d).to(torch.bfloat16), "lse": lse.reshape(n, h)}


def _wprompt_plain(s):
    h, d = s["q"].shape[1:]
    hk = s["k"].shape[1]
    window, sinks, block = s["case"]["window"], s["case"]["sinks"], 1024
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    start = 0
    for m in _lengths(s["case"]):
        k, v = (s[x][start:start + m].float().transpose(0, 1) for x in "kv")  # [kv_heads, m, d]
        for i0 in range(0, m, block):  # a block of rows against the keys that it can see
            i1 = min(m, i0 + block)
            first = max(0, i0 - window + 1)
            keys = torch.arange(i1, device="cuda")
            keys = torch.cat([keys[:min(sinks, first)], keys[first:]])
            i = torch.arange(i0, i1, device="cuda")[:, None]
            hidden = (keys > i) | (keys <= i - window) & (keys >= sinks)
            q = s["q"][start + i0:start + i1].float().view(i1 - i0, hk, h // hk, d).permute(1, 2, 0, 3)
            scores = (q @ k[:, None, keys].transpose(-1, -2)).mul_(s["scale"])
            o, l = _softmax_product(scores.masked_fill_(hidden, -math.inf), v[:, None, keys])
            out[start + i0:start + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, h, d).to(torch.bfloat16)
            lse[start + i0:start + i1] = l.permute(2, 0, 1).reshape(i1 - i0, h)
        start += m
    return {"out": out, "lse": lse}


def _fork_plain(s):
    page = s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    full = (s["lengths"] // page).long()
    column = torch.arange(s["table"].shape[1], device="cuda")
    old = s["table"][parents]
    new = torch.where(column < full[:, None], old, s["table"][children])
    rest = (s["lengths"] % page)[:, None]
    last = full.clamp(max=s["table"].shape[1] - 1)[:, None]
    new.scatter_(1, last, torch.where(rest > 0, s["new_pages"][:, None], new.gather(1, last)))
    s["table"][children] = new
    source, target = old.gather(1, last)[:, 0].long(), s["new_pages"].long()
    copied = (torch.arange(page, device="cuda") < rest)[:, None, :, None]
    for name in ("k_pages", "v_pages"):
        x = _bits(s[name])
        x[target] = torch.where(copied, x[source], x[target])
    return {"table": s["table"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _compact_plain(s):
    total, page = s["k_pages"].shape[0], s["case"]["page"]
    table = s["table"].long()
    inside = torch.arange(table.shape[1], device="cuda") * page < s["lengths"][:, None]
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    used[table[inside]] = True
    live = used.sum()
    number = torch.arange(total, device="cuda")
    source, target = torch.nonzero(used & (number >= live))[:, 0], torch.nonzero(~used & (number < live))[:, 0]
    number[source] = target
    for name in ("k_pages", "v_pages"):
        x = _bits(s[name])
        x[target] = x[source]
    return {"table": torch.where(inside, number[table], table).to(torch.int32), "live": live.to(torch.int32)[None],
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


_PLAIN = {"tree": _tree_plain, "wdecode": _wdecode_plain, "wprompt": _wprompt_plain, "fork": _fork_plain,
          "compact": _compact_plain}


# ---- what a pass cannot do without, and its result in 64 bits ---------------


def _window_pairs(m, window, sinks):
    """Visible (row, key) pairs of a prompt of m rows."""
    i = np.arange(m, dtype=np.int64)
    return int((np.minimum(i + 1, window) + np.clip(i + 1 - window, 0, sinks)).sum())


def work(case):
    h, hk, d, lens = case["heads"], case["kv_heads"], case["dim"], _lengths(case)
    wide = 1 if case.get("cache") == "e4m3" else 2
    row = 2 * wide * hk * d  # a token's rows of keys and values
    if case["op"] == "tree":
        counts = _nodes(case)
        t = sum(counts)
        words = 0 if case["chain"] else -(-case["nodes"] // 64)
        table = 4 * sum(-(-m // case["page"]) for m in lens)
        # of the pairs among the new tokens, those of a chain; a tree's are fewer and depend on the inputs
        pairs = sum(c * m + (c * (c + 1) // 2 if case["chain"] else c) for c, m in zip(counts, lens))
        return {"bytes": sum(lens) * row + t * (4 * d * h + 4 * d * hk + 4 * h + 8 * words) + table + 8 * len(lens),
                "flops": 4 * h * d * pairs}
    if case["op"] == "wdecode":
        seen = sum(min(m, case["window"] + case["sinks"]) for m in lens)
        return {"bytes": seen * row + len(lens) * h * (4 * d + 4) + 4 * (seen // case["page"]) + 4 * len(lens),
                "flops": 4 * seen * h * d}
    if case["op"] == "wprompt":
        t = sum(lens)
        return {"bytes": t * (4 * d * h + 4 * d * hk + 4 * h) + 4 * (len(lens) + 1),
                "flops": 4 * h * d * sum(_window_pairs(m, case["window"], case["sinks"]) for m in lens)}
    page, kids = case["page"], case.get("children")
    if case["op"] == "fork":
        # a parent's rows of its last page read once and written to every child's; the entries
        return {"bytes": sum(m % page * row * (1 + kids) + 4 * -(-m // page) * (1 + kids) + 16 * kids for m in lens),
                "flops": 0}
    rows, _, _, moves = _layout(case)
    return {"bytes": moves * 2 * page * row + 8 * sum(r[2] for r in rows) + 4 * len(rows), "flops": 0}


def _attend64(q, k, v, scale, hidden):
    """One sequence and key-value head in 64 bits: q [group, rows, d], k and v [positions, d], hidden [rows, positions]."""
    x = torch.einsum("gqd,kd->gqk", q, k) * scale
    x = torch.where(hidden, -math.inf, x)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("gqk,kd->gqd", torch.exp(x - lse[..., None]), v), lse


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # copies: nothing is computed
    s = prepare(case, seed)
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case.get("page")
    group = h // hk
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")

    def kept(i, positions, j, name):
        """Rows of the cache of sequence i and head j in 64 bits."""
        pages = s[name + "_pages"]
        number = s["table"][i].long()[positions // page]
        x = _bits(pages)[number, j, positions % page].view(pages.dtype).double()
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][j].double()

    start = 0
    for i, m in enumerate(_lengths(case)):
        if case["op"] == "wprompt":
            window, sinks = case["window"], case["sinks"]
            for j in range(hk):
                k, v = s["k"][start:start + m, j].double(), s["v"][start:start + m, j].double()
                for i0 in range(0, m, 512):
                    i1, a = min(m, i0 + 512), max(0, i0 + 1 - window)
                    pos = torch.cat([torch.arange(min(sinks, a)), torch.arange(a, i1)]).cuda()
                    away = torch.arange(i0, i1, device="cuda")[:, None] - pos
                    hidden = (away < 0) | ((away >= window) & (pos >= sinks)[None, :])
                    rows, mine = slice(start + i0, start + i1), slice(j * group, (j + 1) * group)
                    o, l = _attend64(s["q"][rows, mine].double().transpose(0, 1), k[pos], v[pos], s["scale"], hidden)
                    out[rows, mine], lse[rows, mine] = o.transpose(0, 1), l.t()
            start += m
            continue
        if case["op"] == "tree":
            n = int(s["cu"][i + 1] - s["cu"][i])
            pos = torch.arange(m, device="cuda")
            seen = np.zeros((n, n), dtype=bool)
            if case["chain"]:
                seen = np.tri(n, dtype=bool)
            else:
                bits = s["mask"][start:start + n].cpu().numpy().astype("<i8").view(np.uint8)
                seen = np.unpackbits(bits, axis=1, bitorder="little")[:, :n].astype(bool)
            hidden = torch.cat([torch.zeros((n, m), dtype=torch.bool), torch.from_numpy(~seen)], 1).cuda()
        else:
            n = 1
            pos = torch.tensor([p for p in range(m) if p < case["sinks"] or p >= m - case["window"]], device="cuda")
            hidden = torch.zeros((1, len(pos)), dtype=torch.bool, device="cuda")
        rows = slice(start, start + n)
        for j in range(hk):
            k, v = kept(i, pos, j, "k"), kept(i, pos, j, "v")
            if case["op"] == "tree":
                k, v = torch.cat([k, s["k"][rows, j].double()]), torch.cat([v, s["v"][rows, j].double()])
            mine = slice(j * group, (j + 1) * group)
            o, l = _attend64(s["q"][rows, mine].double().transpose(0, 1), k, v, s["scale"], hidden)
            out[rows, mine], lse[rows, mine] = o.transpose(0, 1), l.t()
        start += n
    return {"out": out, "lse": lse}
