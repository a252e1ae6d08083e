"""A wait bound that runs out in the MXFP4 products becomes MOE_DEV_TIMEOUT in the caller's status word.

As for the other grouped kernels: a child process sets the bound to 1 ns, so the first wait of every role
that is not satisfied at once runs out. Producers, scale warps, MMA issuer and epilogue leave their loops, the
teardown waits (bounded by seconds) for copies and MMAs in flight, tensor memory is freed and the
kernels return; the down product, started as the up product ends, leaves the same way. Two layers in
turn, so that a second call follows an aborted one."""
import os
import subprocess
import sys
import time

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
from ragged_grouped_gemm_device_gb300.layer import Mxfp4ExpertLayer

T, k, E, d, h = 1024, 4, 8, 2048, 1024  # 8 stages a tile of the up product, 4 of the down product
g = torch.Generator("cuda").manual_seed(1)
n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
layer = Mxfp4ExpertLayer(n(E, 2 * h, d) / 45, n(E, h, d) / 32)
for _ in range(2):
    layer.forward(n(T, d), ids, torch.ones(T, k, device="cuda"))
torch.cuda.synchronize()
check = (torch.ones(4096, device="cuda") * 2).sum().item()  # the context is still usable
print("STATUS", layer.status.item(), "CHECK", check, flush=True)
"""


def _run(timeout_ns):
    env = dict(os.environ)
    env.pop("MOE_GG_WAIT_TIMEOUT_NS", None)
    if timeout_ns is not None:
        env["MOE_GG_WAIT_TIMEOUT_NS"] = str(timeout_ns)
    t0 = time.monotonic()
    res = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    line = [ln for ln in res.stdout.splitlines() if ln.startswith("STATUS")][-1].split()
    assert float(line[3]) == 8192.0
    return int(line[1]), time.monotonic() - t0


def test_expired_wait_bound_reports_timeout_and_returns(lib):
    from ragged_grouped_gemm_device_gb300 import _lib
    status, elapsed = _run(1)
    assert status & _lib.MOE_DEV_TIMEOUT, f"status {status}: no wait ran out"
    # four products, each bounded by its teardown waits (seconds), plus process start-up
    assert elapsed < 240, f"took {elapsed:.0f} s"
    assert _run(None)[0] == 0  # with the bound as it is the same program waits long enough
