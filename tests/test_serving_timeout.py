"""A wait that runs out inside the tcgen05 kernel of attention over a cache: the kernel gives up cleanly, the call
reports SDPA_ERR_TIMEOUT, and the context stays usable (a child process shortens the bound to one cycle)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import os, sys
sys.path.insert(0, os.path.join(ROOT, "tests")); sys.path.insert(0, ROOT)
import torch
import attention_flashattention_sdpa_gb300 as m
from oracle import serving_oracle as so
from sdpa_testlib import f64
from serving_testlib import assert_attend_close, kv_rounding, make_cache, randn

for kind, dtype in (("bf16", "bf16"), ("e4m3", "bf16")):
    c = make_cache((700, 300), 2, 128, 16, kind, seed=1)
    g = torch.Generator().manual_seed(2)
    q = randn(g, 2, 20, 4, 128).bfloat16().cuda().permute(0, 2, 1, 3)
    o, lse = torch.empty_like(q), torch.empty(2, 4, 20, device="cuda")
    ws = torch.empty(m.sdpa_decode_workspace_size(q, *c.where(), **c.scales()), dtype=torch.uint8, device="cuda")
    call = lambda: m.sdpa_decode(q, *c.where(), o, lse, workspace=ws, **c.scales(), causal="bottom_right")
    os.environ["SDPA_WAIT_LIMIT_CYCLES"] = "1"
    try:
        call()
        status = 0
    except m.SdpaError as e:
        status = e.status
    assert status == 6, f"{kind}: status {status}, want SDPA_ERR_TIMEOUT"
    assert m.sdpa_device_error() == 0, "the flag is reported once and then cleared"
    del os.environ["SDPA_WAIT_LIMIT_CYCLES"]
    call()
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, (700, 300), None, 128 ** -0.5, True)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, 40, 128, dtype))
print("WAIT_TIMEOUT_OK")
'''


@pytest.mark.gpu
def test_waits_that_run_out_report_a_timeout_and_leave_the_context_usable():
    env = dict(os.environ, SDPA_DEBUG_SYNC="1")
    env.pop("SDPA_WAIT_LIMIT_CYCLES", None)
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + CHILD], env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "WAIT_TIMEOUT_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
