"""A rollout through the attention half of one decoder block: packed prompts in, then one token
per sequence and step.

    python examples/rollout_block.py

Per pass: RMSNorm with the merged noise and the q/k/v linears (NVFP4 weights, LoRA, one launch
group), rotation with the append to the paged cache, attention, the o linear, the residual.
Prompts use causal attention of the packed rows; every later step uses attention of the new token
over the cache and is one CUDA graph, replayed with the positions and lengths updated on the
device.  Weights and hidden states are synthetic.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_weight_quantized_03_gb300 as q  # noqa: E402
import workloads as wl  # noqa: E402


class AttentionHalf:
    """Weights, cache and buffers of the attention half of one block for `seqs` sequences of at most
    `max_len` tokens.  cache_dtype: torch.bfloat16 or torch.float8_e4m3fn."""

    def __init__(self, heads, kv_heads, dim, seqs, max_len, page=16, cache_dtype=torch.bfloat16, rank=16, sigma=1e-2,
                 seed=0):
        self.heads, self.kv_heads, self.dim, self.seqs = heads, kv_heads, dim, seqs
        self.hidden, self.rank, self.scale = heads * dim, rank, 1.0 / math.sqrt(dim)
        dev = "cuda"
        self.weights = {}
        for i, (name, n, k) in enumerate([("q", heads * dim, self.hidden), ("k", kv_heads * dim, self.hidden),
                                          ("v", kv_heads * dim, self.hidden), ("o", self.hidden, heads * dim)]):
            codes, scales, S = q.quantize(wl.weight_f32_device(n, k, seed, i, device=dev))
            self.weights[name] = (q.pack(codes, scales), S, wl.normal_bf16_device((rank, k), k ** -0.5, seed, i, 1),
                                  wl.normal_bf16_device((n, rank), 0.01, seed, i, 2), 2.0 * rank)
        self.norm = (wl.normal_bf16_device((self.hidden,), 0.1, seed, 9) + 1.0).to(torch.bfloat16)
        self.noise = torch.empty(self.hidden, dtype=torch.float32, device=dev)
        q.check(q.qerl_aqn_sample(self.noise, sigma, seed=seed))
        # pages in no particular order, as a server's free list leaves them
        per_seq = -(-max_len // page)
        order = torch.randperm(seqs * per_seq, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        shape = (seqs * per_seq, kv_heads, page, dim)
        pages = [torch.zeros(shape, dtype=torch.bfloat16, device=dev).to(cache_dtype) for _ in range(2)]
        scale = None
        if cache_dtype != torch.bfloat16:  # an 8-bit cache: the largest expected value at 448
            scale = torch.full((kv_heads,), 16.0 / 448, dtype=torch.float32, device=dev)
        self.cache = q.kv_cache(*pages, order.view(seqs, per_seq).cuda(), scale, scale)
        self.inv_freq = (1e6 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))).cuda()
        self.append_ws = q.workspace(q.qerl_rope_append_workspace_size())
        self.decode_ws = q.workspace(q.qerl_decode_attention_workspace_size(seqs, heads, kv_heads, dim))
        self.prompt_ws = []  # one per prompt pass, until its status is read

    def buffers(self, rows):
        """What one pass over `rows` rows writes, allocated once."""
        empty = lambda n: torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
        b = {"q": empty(self.heads * self.dim), "k": empty(self.kv_heads * self.dim), "v": empty(self.kv_heads * self.dim),
             "att": empty(self.heads * self.dim), "o": empty(self.hidden),
             "lse": torch.empty((rows, self.heads), dtype=torch.float32, device="cuda")}
        b["qkv"] = q.linear_descs([(*self.weights[n][:4], self.weights[n][4], b[n]) for n in "qkv"])
        b["ws"] = q.workspace(q.qerl_rmsnorm_lora_linear_group_workspace_size(rows, self.hidden, b["qkv"]))
        b["o_ws"] = q.workspace(q.qerl_lora_linear_workspace_size(rows, self.hidden, self.heads * self.dim, self.rank))
        return b

    def _project(self, h, b, positions, seq_ids):
        """q, k, v of the rows, rotated, k and v in the cache; q and k are rotated in place."""
        q.check(q.qerl_rmsnorm_lora_linear_group(h, self.norm, self.noise, 1e-6, b["qkv"], b["ws"]), "qkv")
        rows = lambda x, n: x.unflatten(1, (n, self.dim))
        qh, kh, vh = rows(b["q"], self.heads), rows(b["k"], self.kv_heads), rows(b["v"], self.kv_heads)
        q.check(q.qerl_rope_append(self.cache, qh, kh, vh, positions, self.inv_freq, qh, kh, self.append_ws, seq_ids),
                "append")
        return qh, kh, vh, rows(b["att"], self.heads)

    def _output(self, h, b):
        wp, S, A, B, alpha = self.weights["o"]
        q.check(q.qerl_lora_linear(b["att"], wp, S, None, A, B, alpha, b["o"], b["o_ws"]), "o")
        return h + b["o"]

    def prompts(self, h, lens):
        """h [sum(lens), hidden]: the packed prompts' hidden states -> the same shape, the cache filled."""
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        positions = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
        seq_ids = torch.repeat_interleave(torch.arange(len(lens), dtype=torch.int32), torch.tensor(lens)).cuda()
        b = self.buffers(h.shape[0])
        qh, kh, vh, att = self._project(h, b, positions, seq_ids)
        ws = q.workspace(q.qerl_prompt_attention_workspace_size(h.shape[0], self.heads, self.kv_heads, self.dim, len(lens)))
        self.prompt_ws.append(ws)
        q.check(q.qerl_prompt_attention(qh, kh, vh, cu.cuda(), self.scale, att, b["lse"], ws), "prompt attention")
        return self._output(h, b)

    def step(self, h, b, lengths):
        """h [seqs, hidden]: one new token per sequence; lengths [seqs] int32 counts it already."""
        qh, kh, vh, att = self._project(h, b, lengths - 1, None)
        q.check(q.qerl_decode_attention(self.cache, qh, lengths, self.scale, att, b["lse"], self.decode_ws), "decode")
        return self._output(h, b)

    def status(self):
        """What the device recorded since the last call: the first error, or QERL_OK.  Synchronises."""
        found = [q.qerl_read_status(w) for w in (self.append_ws, self.decode_ws, *self.prompt_ws)]
        self.prompt_ws.clear()
        return next((s for s in found if s != q.QERL_OK), q.QERL_OK)


def rollout(heads=8, kv_heads=2, dim=128, lens=(37, 5, 130, 64), steps=6, cache_dtype=torch.bfloat16, seed=0):
    """Prompts, then `steps` graph replays.  Returns (every step's output, the same rows from one pass of
    causal attention over the whole sequences, microseconds per replay)."""
    half = AttentionHalf(heads, kv_heads, dim, len(lens), max(lens) + steps, cache_dtype=cache_dtype, seed=seed)
    total = [m + steps for m in lens]
    hidden = wl.normal_bf16_device((sum(total), half.hidden), 1.0, seed, 77)  # what the layers below would give
    start = [sum(total[:i]) for i in range(len(lens))]
    half.prompts(torch.cat([hidden[s:s + m] for s, m in zip(start, lens)]), list(lens))

    b = half.buffers(len(lens))
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    h = torch.zeros((len(lens), half.hidden), dtype=torch.bfloat16, device="cuda")
    run = torch.cuda.Stream()
    run.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=run):
        lengths += 1
        out = half.step(h, b, lengths)
    got = []
    for t in range(steps):
        h.copy_(torch.stack([hidden[s + m + t] for s, m in zip(start, lens)]))
        graph.replay()
        got.append(out.clone())
    q.check(half.status(), "prompts and steps")

    whole = half.prompts(hidden, total)
    q.check(half.status(), "the whole sequences")
    want = [torch.stack([whole[s + m + t] for s, m in zip(start, lens)]) for t in range(steps)]
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    lengths -= steps  # the timed replays write the same rows again
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return got, want, begin.elapsed_time(end) / steps * 1e3


if __name__ == "__main__":
    for dtype in (torch.bfloat16, torch.float8_e4m3fn):
        got, want, us = rollout(cache_dtype=dtype)
        far = max(((a.float() - b.float()).norm() / b.float().norm()).item() for a, b in zip(got, want))
        print(f"{str(dtype):22s} {len(got)} steps, {us:.1f} us each; against one causal pass: {far:.2e} (relative norm)")
