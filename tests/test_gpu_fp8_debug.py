"""The FP8 calls under the debug build (libpact_debug.so): their tests pass with every
index check on and none failing, and a NaN or an infinity, which these calls take, is no
error that pact_check_status reports."""
import os
import subprocess
import sys

import pytest

from nvfp4_frozen_projection_gb300 import build as pact_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

# Every FP8 entry point with a NaN and with infinities, in a row of its own: the status
# word stays clear, the row is NaN where the contract says so and the others are untouched.
NON_FINITE = """
import torch
import nvfp4_frozen_projection_gb300 as pk
assert pk.library_path().endswith("libpact_debug.so"), pk.library_path()
torch.manual_seed(0)
M, K, N, row = 300, 272, 144, 77
keep = torch.arange(M, device="cuda") != row
cols = torch.arange(K, device="cuda") != 9
x = torch.randn(M, K, device="cuda").bfloat16()
gamma = (1 + 0.1 * torch.randn(K, device="cuda")).bfloat16()
dy = torch.randn(M, K, device="cuda").bfloat16()
W = 0.05 * torch.randn(N, K, device="cuda")
w = pk.pact_pack_weight_fp8_fwd(W)

def products(x):
    xq, (_, yq, _) = pk.pact_quant_fp8(x), pk.pact_add_rmsnorm_quant_fp8(x, None, gamma)
    return pk.pact_linear_fp8_fwd(xq, w), pk.pact_linear_fp8_fwd(yq, w)

rstd = pk.pact_add_rmsnorm_quant_fp8(x, None, gamma)[2]
base, (dh0, dg0) = products(x), pk.pact_add_rmsnorm_bwd(x, gamma, rstd, dy, dgamma=True)
pk.pact_check_status()
for bad in (float("nan"), float("inf"), float("-inf")):
    xb = x.clone()
    xb[row, 5] = bad
    for y, y0 in zip(products(xb), base):
        assert bool(torch.isnan(y[row]).all()) and torch.equal(y[keep], y0[keep])
    hb, _, _ = pk.pact_add_rmsnorm_quant_fp8(xb, x, gamma)
    assert not bool(torch.isfinite(hb[row, 5]))
    wb = W.clone()
    wb[3, 40] = bad
    for q in (pk.pact_pack_weight_fp8_fwd(wb).q, pk.pact_pack_weight_fp8_bwd(wb).q.t()):
        assert bool(torch.isnan(q[3, 40].float()))
    pk.pact_check_status()
    db = dy.clone()
    db[row, 9] = bad
    dh, dg = pk.pact_add_rmsnorm_bwd(x, gamma, rstd, db, dgamma=True)
    assert not bool(torch.isfinite(dh[row]).any()) and torch.equal(dh[keep], dh0[keep])
    assert not bool(torch.isfinite(dg[9])) and torch.equal(dg[cols], dg0[cols])
    pk.pact_check_status()
print("non-finite values ok")
"""


@pytest.fixture(scope="module")
def debug_env():
    pact_build.build_debug()
    env = dict(os.environ, PACT_DEBUG="1")
    env["PYTHONPATH"] = os.pathsep.join(p for p in (ROOT, env.get("PYTHONPATH")) if p)
    return env


def test_non_finite_values_are_no_error(debug_env):
    r = subprocess.run([sys.executable, "-c", NON_FINITE], env=debug_env, cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "non-finite values ok" in r.stdout


def test_fp8_suite_under_the_debug_build(debug_env):
    # two cases of tens of gigabytes are left to the release build
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu",
                        "-k", "not past_32_bits", os.path.join(HERE, "test_gpu_fp8.py")],
                       env=debug_env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
