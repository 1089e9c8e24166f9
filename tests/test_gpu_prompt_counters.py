"""The prompt attention's running counters pass 2^31 and 2^32 without a trace.

A CTA counts its loads and steps over all its items; calls long enough to wrap would take hours.  The
test-only build (QERL_TEST_HOOKS) lets the counters begin shortly before the wraps.  Run in a subprocess
with its own copy of the library."""
import json
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

_SCRIPT = r"""
import ctypes, json, os, sys
import torch
sys.path.insert(0, os.environ["QERL_ROOT"])
import nvfp4_weight_quantized_03_gb300 as q
from nvfp4_weight_quantized_03_gb300 import build
q._build.LIB = build.build(test_hooks=True)
L = q.lib()
L.qerl_test_set_prompt_first_count.restype = ctypes.c_int
L.qerl_test_set_prompt_first_count.argtypes = [ctypes.c_uint]
assert L.qerl_test_set_prompt_first_count(8) == 1
out = []
for dim, heads, hk in ((64, 40, 8), (128, 40, 8)):
    g = torch.Generator(device="cuda").manual_seed(dim)
    lens = [1500, 90, 2300, 129, 256]
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    t = sum(lens)
    x = [torch.randn((t, h, dim), generator=g, device="cuda").to(torch.bfloat16) for h in (heads, hk, hk)]
    ws = q.workspace(q.qerl_prompt_attention_workspace_size(t, heads, hk, dim, len(lens)))
    want = None
    for first in (0, 2 ** 31 - 16, 2 ** 31 - 64, 2 ** 32 - 16, 2 ** 32 - 32, 2 ** 32 - 96):
        assert L.qerl_test_set_prompt_first_count(first) == 0
        o, lse = torch.full_like(x[0], 5.0), torch.full((t, heads), 5.0, device="cuda")
        call = q.qerl_prompt_attention(*x, cu, 0.1, o, lse, ws)
        status = q.qerl_read_status(ws)
        want = want or (o, lse)
        out.append([dim, first, call, status, bool(torch.equal(o, want[0]) and torch.equal(lse, want[1])),
                    bool(torch.isfinite(o.float()).all() and (lse != 5.0).all())])
print(json.dumps(out))
"""


def test_counters_pass_their_wraps(tmp_path):
    script = tmp_path / "prompt_counters.py"
    script.write_text(_SCRIPT)
    env = dict(os.environ, QERL_ROOT=str(ROOT))
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=600, cwd=ROOT, env=env)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads([l for l in r.stdout.splitlines() if l.startswith("[")][-1])
    assert len(res) == 12
    for dim, first, call, status, same, sound in res:
        assert call == 0 and status == 0 and same and sound, (dim, first, call, status, same, sound)
