"""Backward calls that the host refuses late, by fault injection on the host: the
documented status, nothing enqueued (workspace and gradients keep what they held), and
a context that goes on computing.  As tests/test_host_faults_gpu.py, in a child
process per case; no GPU fault, trap or hang is involved."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, torch
sys.path.insert(0, {root!r})
import scaled_dot_product_13_b200 as sdpa
sdpa.load_library()
B, Hq, Hkv, L, D = 1, 4, 2, 200, {dim}
g = torch.Generator("cpu").manual_seed(1)
q, k, v, out, dout = (torch.randn(B, h, L, D, generator=g).{dtype}().cuda() for h in (Hq, Hkv, Hkv, Hq, Hq))
lse = torch.full((B, Hq, L), 3.0, device="cuda")
d = dict(dq=torch.full_like(q, 7), dk=torch.full_like(k, 7), dv=torch.full_like(v, 7))
n = sdpa.backward_workspace_bytes(B, Hq, Hkv, L, L, D, D, dtype="{name}")
ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
pool = {pool}
try:
    if pool:
        sdpa.backward(q, k, v, out, lse, dout, stream=torch.cuda.current_stream(), **d)
    else:
        sdpa.backward(q, k, v, out, lse, dout, workspace=ws, **d)
    print("STATUS 0")
except sdpa.SdpaError as e:
    print("STATUS", e.status)
    print("MESSAGE", e.message)
torch.cuda.synchronize()
print("UNTOUCHED", all(bool((t == 7).all()) for t in d.values()) and bool((ws == 255).all()))
if pool:  # a workspace of the caller's needs no allocation
    sdpa.backward(q, k, v, out, lse, dout, workspace=ws, **d)
sdpa.device_status()
print("AFTER", bool(torch.isfinite((q @ k.repeat_interleave(2, 1).transpose(2, 3)).float()).all()))
"""


def _run(env, pool, dim, dtype):
    code = CHILD.format(root=ROOT, pool=pool, dim=dim, dtype={"bf16": "bfloat16", "f16": "half"}[dtype], name=dtype)
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, **env}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_kernel_that_does_not_fit(cuda_lib, dim, dtype):
    got = _run({"SDPA_TEST_SMEM_LIMIT": "1024"}, False, dim, dtype)
    assert got["STATUS"] == "3" and "bwd_tc_kernel" in got["MESSAGE"]
    assert got["UNTOUCHED"] == "True" and got["AFTER"] == "True"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_no_memory_for_the_workspace(cuda_lib, dtype):
    got = _run({"SDPA_TEST_FAIL_ALLOC": "1"}, True, 64, dtype)
    assert got["STATUS"] == "4" and "backward workspace" in got["MESSAGE"]
    assert got["UNTOUCHED"] == "True" and got["AFTER"] == "True"
