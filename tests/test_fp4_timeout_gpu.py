"""The bounded waits of the 4-bit products, without a fault: as for the ternary
GEMV, a child process has the first product skip the request of one stage
(BITNET_TEST_STALL=2 the kernel for few tokens, 3 the one for more).  Each wait
on it gives up after its limit (1 s), the kernel frees what it holds and
returns, the status says so once, and the next product is right."""
import json
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

CHILD = r"""
import json, sys, time
import torch
sys.path.insert(0, ROOT)
import ternary_weight_bit_w2a8_b200 as bn
M, N, K, fused = ARGS
gen = torch.Generator().manual_seed(3)
W = (torch.randn(N, K, generator=gen) * 0.02).cuda()
x = torch.randn(M, K, generator=gen).to(torch.bfloat16).cuda()
w, ws = bn.bitnet_fp4_quant(W, bn.BITNET_FP4_NV)
a, sa = bn.bitnet_fp4_quant(x, bn.BITNET_FP4_NV)
def product():
    if fused:
        return bn.bitnet_fp4_linear(x, w, ws, bn.BITNET_FP4_NV)
    return bn.bitnet_fp4_gemm(a, sa, w, ws, K, bn.BITNET_FP4_NV)
t0 = time.time()
product()                                    # the stalled launch
status = bn.bitnet_get_device_error()
dt = time.time() - t0
again = bn.bitnet_get_device_error()         # cleared by the first read
y = product().double()
ref = (bn.bitnet_fp4_dequant(a, sa, K, 1, dtype=torch.float32).double()
       @ bn.bitnet_fp4_dequant(w, ws, K, 1, dtype=torch.float32).double().t())
right = bool(((y - ref).abs() <= ref.abs() / 256 + 1e-4).all())
print(json.dumps({"status": status, "again": again, "right_after": right, "seconds": dt,
                  "final": bn.bitnet_get_device_error()}))
"""


# one CTA per tile; a cluster; tokens quantised in the launch; the pair kernel, four pairs to a tile and one
@pytest.mark.parametrize("stall,args", [("2", (20, 300, 700, 0)), ("2", (1, 600, 6912, 0)), ("2", (3, 600, 6912, 1)),
                                        ("3", (200, 200, 5120, 0)), ("3", (300, 9000, 512, 0))])
def test_bounded_wait_reports_timeout_and_context_survives(stall, args):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_weight_bit_w2a8_b200 as bn
    env = dict(os.environ, BITNET_TEST_STALL=stall)
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\nARGS = {args!r}\n" + CHILD], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["status"] == bn.BITNET_ERR_DEVICE_TIMEOUT
    assert res["again"] == bn.BITNET_OK
    assert res["right_after"]
    assert res["final"] == bn.BITNET_OK
    assert 0.5 < res["seconds"] < 60
