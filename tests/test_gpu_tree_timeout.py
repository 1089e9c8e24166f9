"""A bounded wait of the tree attention that runs out: the call comes back with the status set and
the next call is right.

The test-only build (QERL_TEST_HOOKS) shortens the wait limit to about 1 ms and lets the barriers that
announce the softmax weights expect one arrival that never comes.  Every product issued by then and
every copy completes, so nothing is left in flight when the roles give up; what the outputs then hold is not
specified.
Run in a subprocess with its own copy of the library."""
import json
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

_SCRIPT = r"""
import ctypes, json, os, sys, time
import torch
sys.path.insert(0, os.environ["QERL_ROOT"])
sys.path.insert(0, os.path.join(os.environ["QERL_ROOT"], "tests"))
import nvfp4_weight_quantized_03_gb300 as q
from nvfp4_weight_quantized_03_gb300 import build
from masked_reference import masked64
q._build.LIB = build.build(test_hooks=True)
L = q.lib()
L.qerl_test_set_tree_hooks.restype = ctypes.c_int
L.qerl_test_set_tree_hooks.argtypes = [ctypes.c_longlong, ctypes.c_int]
out = {}
for dim, dtype in ((64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")):
    g = torch.Generator(device="cuda").manual_seed(dim)
    lens, counts = [700, 90], [9, 70]  # rows that both query tiles share, and rows of two tiles
    t = sum(counts)
    x = [torch.randn((t, h, dim), generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2)]
    pages = [torch.randn((13, 2, 64, dim), generator=g, device="cuda").clamp(-4, 4) for _ in range(2)]
    pages = [p.to(torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn) for p in pages]
    table = torch.tensor([list(range(11)), [11, 12] + [0] * 9], dtype=torch.int32, device="cuda")
    cache = q.kv_cache(*pages, table)
    cu, lengths = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 9, 79], lens))
    o, lse = torch.full_like(x[0], 5.0), torch.full((t, 4), 5.0, device="cuda")
    ws = q.workspace(q.qerl_tree_attention_workspace_size(t, 4, 2, dim, 2))
    assert L.qerl_test_set_tree_hooks(2_000_000, 1) == 0
    torch.cuda.synchronize()
    t0 = time.time()
    call = q.qerl_tree_attention(cache, *x, cu, lengths, None, 0.1, o, lse, ws)
    status = q.qerl_read_status(ws)
    seconds = time.time() - t0
    assert L.qerl_test_set_tree_hooks(4_000_000_000, 0) == 0
    call2 = q.qerl_tree_attention(cache, *x, cu, lengths, None, 0.1, o, lse, ws)
    status2 = q.qerl_read_status(ws)
    worst = 0.0
    for s, (a, b) in enumerate(((0, 9), (9, 79))):
        rows = [p.view(torch.uint8 if dtype == "e4m3" else torch.bfloat16)[table[s].long()].view(p.dtype).double() for p in pages]
        rows = [p.transpose(1, 2).reshape(-1, 2, dim)[:lens[s]] for p in rows]
        keep = torch.ones((b - a, lens[s] + b - a), dtype=torch.bool, device="cuda").tril(lens[s])
        for h in range(4):
            k, v = (torch.cat([p[:, h // 2], y[a:b, h // 2].double()]) for p, y in zip(rows, x[1:]))
            w, l, to, tl = masked64(x[0][a:b, h], k, v, 0.1, keep, "bf16")
            worst = max(worst, ((o[a:b, h].double() - w).abs() / to).max().item(),
                        ((lse[a:b, h].double() - l).abs() / tl).max().item())
    out[dtype + str(dim)] = {"call": call, "status": status, "seconds": seconds, "call2": call2, "status2": status2,
                             "worst": worst}
print(json.dumps(out))
"""


def test_bounded_wait_runs_out_and_the_next_call_is_right(tmp_path):
    script = tmp_path / "tree_timeout.py"
    script.write_text(_SCRIPT)
    env = dict(os.environ, QERL_ROOT=str(ROOT))
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=600, cwd=ROOT, env=env)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads([l for l in r.stdout.splitlines() if l.startswith("{")][-1])
    for dim, c in res.items():
        assert c["call"] == 0 and c["status"] == 5, (dim, c)  # launched; QERL_ERR_TIMEOUT recorded
        assert c["seconds"] < 5.0, (dim, c)
        assert c["call2"] == 0 and c["status2"] == 0 and c["worst"] <= 1.0, (dim, c)
