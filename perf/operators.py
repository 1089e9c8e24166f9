"""What the attention operators next to the quantized linears are measured on.

One rollout step runs, between the q/k/v linears and the o linear of a decoder block:

  append  rotates q and k to their positions and writes k and v into the paged cache
  decode  attention of one new token per sequence over the paged cache
  prompt  causal attention of packed whole prompts (the step that fills the cache)

`own` False computes each in its plain form (elementary torch operations, 32-bit arithmetic,
64-bit angles, one rounding at the end); `own` True calls the library's kernels.
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
        # One rollout, one new token: what a single interactive request waits for.
        {"name": "append-one-token", "op": "append", "heads": 16, "kv_heads": 2, "dim": 128, "rot": 128, "cache": "bf16",
         "page": 16, "seqs": 1, "max_len": 700, "prompt": False},
        # A batch of rollouts at far positions, 8-bit cache.
        {"name": "append-batch-e4m3", "op": "append", "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "cache": "e4m3",
         "page": 64, "seqs": 96, "max_len": 131072, "prompt": False},
        # Packed prompts (odd lengths) entering the cache.
        {"name": "append-prompts", "op": "append", "heads": 28, "kv_heads": 4, "dim": 128, "rot": 128, "cache": "bf16",
         "page": 16, "seqs": 9, "max_len": 2731, "prompt": True},
        # One rollout's new token over a short answer.
        {"name": "decode-one", "op": "decode", "heads": 28, "kv_heads": 4, "dim": 128, "cache": "bf16", "page": 16,
         "seqs": 1, "max_len": 777, "ragged": False},
        # One rollout over a long context: few rows, the axis to split.
        {"name": "decode-one-long", "op": "decode", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64,
         "seqs": 1, "max_len": 100003, "ragged": False},
        # A batch of rollouts that are at different lengths.
        {"name": "decode-ragged", "op": "decode", "heads": 28, "kv_heads": 4, "dim": 128, "cache": "bf16", "page": 16,
         "seqs": 64, "max_len": 8192, "ragged": True},
        # Many rollouts in step over an 8-bit cache: the cache fills the card's memory traffic.
        {"name": "decode-batch-e4m3", "op": "decode", "heads": 40, "kv_heads": 8, "dim": 128, "cache": "e4m3", "page": 32,
         "seqs": 128, "max_len": 6000, "ragged": False},
        # Small heads, many short rollouts.
        {"name": "decode-small-heads", "op": "decode", "heads": 32, "kv_heads": 8, "dim": 64, "cache": "bf16", "page": 24,
         "seqs": 256, "max_len": 1500, "ragged": True},
        # One short prompt: latency.
        {"name": "prompt-short", "op": "prompt", "heads": 28, "kv_heads": 4, "dim": 128, "seqs": 1, "max_len": 77,
         "ragged": False},
        # A batch of prompts of different lengths, packed.
        {"name": "prompt-packed", "op": "prompt", "heads": 28, "kv_heads": 4, "dim": 128, "seqs": 12, "max_len": 3001,
         "ragged": True},
        # One long prompt: arithmetic bound.
        {"name": "prompt-long", "op": "prompt", "heads": 40, "kv_heads": 8, "dim": 128, "seqs": 1, "max_len": 8192,
         "ragged": False},
        # Small heads, packed.
        {"name": "prompt-small-heads", "op": "prompt", "heads": 32, "kv_heads": 8, "dim": 64, "seqs": 5, "max_len": 4500,
         "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    heads, kv_heads, dim = rng.choice(_BLOCKS)
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim}
    if op == "append":
        prompt = rng.random() < 0.5
        case |= {"rot": rng.choice([dim, dim, dim // 2]), "cache": rng.choice(["bf16", "e4m3"]), "page": rng.choice(_PAGES),
                 "prompt": prompt}
        case |= ({"seqs": _log_int(rng, 1, 12), "max_len": _log_int(rng, 1, 2500)} if prompt else
                 {"seqs": _log_int(rng, 1, 512), "max_len": _log_int(rng, 1, 131072)})
        if not prompt and case["page"] < 8:
            case["page"] = 8
    elif op == "decode":
        seqs = _log_int(rng, 1, 256)
        case |= {"cache": rng.choice(["bf16", "e4m3"]), "page": rng.choice(_PAGES), "seqs": seqs,
                 "max_len": _log_int(rng, 1, min(100000, 400000 // seqs)), "ragged": rng.random() < 0.6}
    else:
        seqs = _log_int(rng, 1, 16)
        most = min(20000 // seqs, int(math.sqrt(40 * 8192 ** 2 / (heads * seqs))), 8192)  # no dearer than the longest prompt
        case |= {"seqs": seqs, "max_len": _log_int(rng, 1, most), "ragged": rng.random() < 0.6}
    return case


def _lengths(case):
    """The sequences' lengths: the longest first or last, the others spread over the logarithm of the range."""
    n, longest = case["seqs"], case["max_len"]
    if not case.get("ragged", case["op"] == "append"):
        return [longest] * n
    r = random.Random("%d %d" % (n, longest))
    lens = [_log_int(r, max(1, longest // 16), longest) for _ in range(n)]
    lens[r.randrange(n)] = longest
    return lens


def _normal(shape, g, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _cache(case, lens, g, fill):
    """Key and value pages, the sequences' page table (pages in no order, unused entries 0) and the
    scales of an 8-bit cache. `fill` False: only every sequence's last page is its own, the earlier ones
    are shared (rollouts of one prompt), as appending touches the last alone."""
    page, n = case["page"], len(lens)
    used = [-(-m // page) for m in lens]
    own_pages = used if fill else [1] * n
    total = sum(own_pages) + (0 if fill else 4)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table = np.zeros((n, max(used)), dtype=np.int32)
    at = 0
    for i in range(n):
        if not fill:
            table[i, :used[i]] = order[np.arange(used[i]) % 4 - 4]
        table[i, used[i] - own_pages[i]:used[i]] = order[at:at + own_pages[i]]
        at += own_pages[i]
    shape = (total, case["kv_heads"], page, case["dim"])
    e4m3 = case["cache"] == "e4m3"
    s = {"table": torch.from_numpy(table).cuda()}
    for name in ("k", "v"):
        pages = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        pages.normal_(generator=g)
        if e4m3:
            # an 8-bit cache holds value / scale, with the scales set from the values' largest
            s[name + "_scale"] = torch.rand(case["kv_heads"], generator=g, device="cuda") * 0.01 + 0.008
            pages = (pages.float() / s[name + "_scale"][:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            s[name + "_scale"] = None
        s[name + "_pages"] = pages
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    n = len(lens)
    s = {"case": case}
    if case["op"] == "append":
        whole = case["prompt"]
        s |= _cache(case, lens, g, fill=whole)
        tokens = sum(lens) if whole else n
        if whole:
            s["positions"] = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
            s["seq_ids"] = torch.repeat_interleave(torch.arange(n, dtype=torch.int32), torch.tensor(lens)).cuda()
        else:
            s["positions"] = torch.tensor([m - 1 for m in lens], dtype=torch.int32).cuda()
            s["seq_ids"] = torch.arange(n, dtype=torch.int32).cuda()
        s["q"], s["k"], s["v"] = _normal((tokens, h, d), g), _normal((tokens, hk, d), g), _normal((tokens, hk, d), g)
        half = case["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).cuda()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif case["op"] == "decode":
        s |= _cache(case, lens, g, fill=True)
        s["q"] = _normal((n, h, d), g, 1.5)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((n, h), device="cuda")
    else:
        tokens = sum(lens)
        s["q"], s["k"], s["v"] = _normal((tokens, h, d), g, 1.5), _normal((tokens, hk, d), g), _normal((tokens, hk, d), g)
        s["cu_seqlens"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((tokens, h), device="cuda")
    s["scale"] = 1.0 / math.sqrt(d)
    if own:  # the cache's descriptor and the workspace, made once and kept
        import nvfp4_weight_quantized_03_gb300 as q
        if "k_pages" in s:
            s["cache"] = q.kv_cache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"])
        s["ws"] = q.workspace(q.qerl_rope_append_workspace_size() if case["op"] == "append" else
                              q.qerl_decode_attention_workspace_size(n, h, hk, d) if case["op"] == "decode" else
                              q.qerl_prompt_attention_workspace_size(tokens, h, hk, d, n))
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "decode": _decode_own, "prompt": _prompt_own}[op](state)
    return {"append": _append_plain, "decode": _decode_plain, "prompt": _prompt_plain}[op](state)


# ---- the library's calls ----------------------------------------------------


def _append_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_rope_append(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["q_out"],
                               s["k_out"], s["ws"], seq_ids=s["seq_ids"]))
    return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _decode_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_decode_attention(s["cache"], s["q"], s["lengths"], s["scale"], s["out"], s["lse"], s["ws"]))
    return {"out": s["out"], "lse": s["lse"]}


def _prompt_own(s):
    import nvfp4_weight_quantized_03_gb300 as q
    q.check(q.qerl_prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["scale"], s["out"], s["lse"], s["ws"]))
    return {"out": s["out"], "lse": s["lse"]}


# ---- the plain forms --------------------------------------------------------


def _rotate(x, cos, sin):
    """The pair (x[i], x[i + half]) turned by its angle; columns past the rotated ones stay."""
    half = cos.shape[-1]
    a, b, rest = x[..., :half].float(), x[..., half:2 * half].float(), x[..., 2 * half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)


def _store(pages, at, rows, scale):
    """Writes rows [tokens, kv_heads, dim] (fp32) to pages[page, :, row] in the pages' type."""
    if pages.dtype == torch.bfloat16:
        pages[at[0], :, at[1]] = rows.to(torch.bfloat16)
    else:
        bits = (rows / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pages.view(torch.uint8)[at[0], :, at[1]] = bits


def _append_plain(s):
    pos, page = s["positions"].long(), s["case"]["page"]
    angle = pos.double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q, k = _rotate(s["q"], cos, sin), _rotate(s["k"], cos, sin)
    at = (s["table"][s["seq_ids"].long(), pos // page].long(), pos % page)
    _store(s["k_pages"], at, k, s["k_scale"])
    _store(s["v_pages"], at, s["v"].float(), s["v_scale"])
    return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _gathered(pages, table, scale):
    """[seqs, kv_heads, positions, dim] in fp32, in the order of the sequences' positions."""
    x = pages.view(torch.uint8)[table.long()].view(pages.dtype) if pages.dtype != torch.bfloat16 else pages[table.long()]
    x = x.float().permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _softmax_product(scores, v):
    """(softmax(scores) v, log sum exp): scores [..., rows, positions] with -inf where masked."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total, (total.log() + top)[..., 0]


def _decode_plain(s):
    n, h, d = s["q"].shape
    k, v = _gathered(s["k_pages"], s["table"], s["k_scale"]), _gathered(s["v_pages"], s["table"], s["v_scale"])
    hk = k.shape[1]
    scores = (s["q"].float().view(n, hk, h // hk, d) @ k.transpose(-1, -2)) * s["scale"]
    past = torch.arange(k.shape[2], device="cuda") >= s["lengths"][:, None]
    out, lse = _softmax_product(scores.masked_fill(past[:, None, None, :], -math.inf), v)
    return {"out": out.reshape(n, h, d).to(torch.bfloat16), "lse": lse.reshape(n, h)}


def _prompt_plain(s):
    t, h, d = s["q"].shape
    hk = s["k"].shape[1]
    n, longest = s["case"]["seqs"], s["case"]["max_len"]
    # the packed rows laid out as [sequences, longest], then back
    cu = s["cu_seqlens"].long()
    row = torch.arange(t, device="cuda")
    seq = torch.bucketize(row, cu[1:], right=True)
    at = seq * longest + row - cu[seq]

    def padded(x):
        full = torch.zeros((n * longest,) + x.shape[1:], device="cuda")
        full[at] = x.float()
        return full.view(n, longest, hk, -1, d).permute(0, 2, 3, 1, 4)  # [n, kv_heads, group, longest, d]

    scores = padded(s["q"]) @ padded(s["k"]).transpose(-1, -2)
    scores.mul_(s["scale"])
    later = torch.ones((longest, longest), dtype=torch.bool, device="cuda").triu(1)
    out, lse = _softmax_product(scores.masked_fill_(later, -math.inf), padded(s["v"]))
    out = out.permute(0, 3, 1, 2, 4).reshape(n * longest, h, d)[at]
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(n * longest, h)[at]}


# ---- what a pass cannot do without, and its result in 64 bits ---------------


def work(case):
    h, hk, d, lens = case["heads"], case["kv_heads"], case["dim"], _lengths(case)
    wide = 1 if case.get("cache") == "e4m3" else 2
    if case["op"] == "append":
        t = sum(lens) if case["prompt"] else len(lens)
        # q, k, v in; q, k out; the cache's rows; positions, sequence ids, page numbers
        return {"bytes": t * (2 * d * (h + 2 * hk) + 2 * d * (h + hk) + 2 * wide * d * hk + 12) + 4 * case["rot"],
                "flops": t * (h + hk) * 3 * case["rot"]}
    if case["op"] == "decode":
        live = sum(lens)
        table = 4 * sum(-(-m // case["page"]) for m in lens)
        return {"bytes": 2 * live * hk * d * wide + len(lens) * h * (4 * d + 4) + table + 4 * len(lens),
                "flops": 4 * live * h * d}
    t = sum(lens)
    return {"bytes": t * (4 * d * h + 4 * d * hk + 4 * h) + 4 * (len(lens) + 1),
            "flops": 4 * h * d * sum(m * (m + 1) // 2 for m in lens)}


def _attend64(q, k, v, scale, causal):
    """One sequence and key-value head in 64 bits: q [group, rows, d], k and v [positions, d]."""
    x = torch.einsum("gqd,kd->gqk", q, k) * scale
    if causal:
        x = torch.where(torch.ones(x.shape[1:], dtype=torch.bool, device=x.device).tril(), x, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("gqk,kd->gqd", torch.exp(x - lse[..., None]), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case.get("page")
    lens, group = _lengths(case), case["heads"] // case["kv_heads"]
    if case["op"] == "append":
        half = case["rot"] // 2
        pos = s["positions"].double()
        turn = torch.polar(torch.ones((pos.numel(), half), dtype=torch.float64, device="cuda"),
                           torch.outer(pos, s["inv_freq"]))[:, None, :]
        got = {}
        for name in ("q", "k"):
            x = s[name].double()
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
            got[name] = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
        number = s["table"].long()[s["seq_ids"].long(), s["positions"].long() // page]
        for name, rows in (("k_pages", got["k"]), ("v_pages", s["v"].double())):
            full = s[name].double()
            scale = s[name[0] + "_scale"]
            rows = rows if scale is None else (rows / scale.double()[:, None]).clamp(-448, 448)
            full[number, :, s["positions"].long() % page] = rows
            got[name] = full
        return got
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    start = 0
    for i, m in enumerate(lens):
        rows = slice(start, start + m) if case["op"] == "prompt" else slice(i, i + 1)
        start += m
        for j in range(hk):
            mine = slice(j * group, (j + 1) * group)
            if case["op"] == "prompt":
                k, v = s["k"][rows, j].double(), s["v"][rows, j].double()
            else:
                used = s["table"][i, :-(-m // page)].long()
                k, v = (s[x + "_pages"].view(torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16)[used, j]
                        .view(s[x + "_pages"].dtype).reshape(-1, d)[:m].double() for x in "kv")
                if case["cache"] == "e4m3":
                    k, v = k * s["k_scale"][j].double(), v * s["v_scale"][j].double()
            o, l = _attend64(s["q"][rows, mine].double().transpose(0, 1), k, v, s["scale"], case["op"] == "prompt")
            out[rows, mine], lse[rows, mine] = o.transpose(0, 1), l.t()
    return {"out": out, "lse": lse}
