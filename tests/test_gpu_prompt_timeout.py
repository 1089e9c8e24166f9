"""A bounded wait of the prompt attention that runs out: the call comes back with the status set and
the next call is right.

The test-only build (QERL_TEST_HOOKS) shortens the wait limit to about 1 ms and lets the barriers that
announce the softmax weights expect one arrival that never comes.  Every product issued by then and
every copy completes, so nothing is left in flight when the roles give up; the outputs are not written.
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
from attention_reference import causal64
q._build.LIB = build.build(test_hooks=True)
L = q.lib()
L.qerl_test_set_prompt_hooks.restype = ctypes.c_int
L.qerl_test_set_prompt_hooks.argtypes = [ctypes.c_longlong, ctypes.c_int]
out = {}
for dim in (64, 128):
    g = torch.Generator(device="cuda").manual_seed(dim)
    lens = [700, 90, 300]
    t = sum(lens)
    x = [torch.randn((t, h, dim), generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2)]
    cu = torch.tensor([0, 700, 790, 1090], dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(x[0], 5.0), torch.full((t, 4), 5.0, device="cuda")
    ws = q.workspace(q.qerl_prompt_attention_workspace_size(t, 4, 2, dim, 3))
    assert L.qerl_test_set_prompt_hooks(2_000_000, 1) == 0
    torch.cuda.synchronize()
    t0 = time.time()
    call = q.qerl_prompt_attention(*x, cu, 0.1, o, lse, ws)
    status = q.qerl_read_status(ws)
    seconds = time.time() - t0
    untouched = bool((o == 5).all().item())
    assert L.qerl_test_set_prompt_hooks(4_000_000_000, 0) == 0
    call2 = q.qerl_prompt_attention(*x, cu, 0.1, o, lse, ws)
    status2 = q.qerl_read_status(ws)
    worst = 0.0
    for a, b in ((0, 700), (700, 790), (790, 1090)):
        for h in range(4):
            w, l, to, tl = causal64(x[0][a:b, h], x[1][a:b, h // 2], x[2][a:b, h // 2], 0.1, "bf16")
            worst = max(worst, ((o[a:b, h].double() - w).abs() / to).max().item(),
                        ((lse[a:b, h].double() - l).abs() / tl).max().item())
    out[dim] = {"call": call, "status": status, "seconds": seconds, "untouched": untouched, "call2": call2,
                "status2": status2, "worst": worst}
print(json.dumps(out))
"""


def test_bounded_wait_runs_out_and_the_next_call_is_right(tmp_path):
    script = tmp_path / "prompt_timeout.py"
    script.write_text(_SCRIPT)
    env = dict(os.environ, QERL_ROOT=str(ROOT))
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=600, cwd=ROOT, env=env)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads([l for l in r.stdout.splitlines() if l.startswith("{")][-1])
    for dim, c in res.items():
        assert c["call"] == 0 and c["status"] == 5, (dim, c)  # launched; QERL_ERR_TIMEOUT recorded
        assert c["seconds"] < 5.0 and c["untouched"], (dim, c)
        assert c["call2"] == 0 and c["status2"] == 0 and c["worst"] <= 1.0, (dim, c)
