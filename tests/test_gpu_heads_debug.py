"""The operators on heads, attention and gradient clipping under the debug build
(libpact_debug.so): their tests pass with every index check on and none failing.  A NaN or an
infinity, which these calls take, is no error there."""
import os
import subprocess
import sys

import pytest

from nvfp4_frozen_projection_gb300 import build as pact_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.parametrize("name", ["test_gpu_rope.py", "test_gpu_attention.py", "test_gpu_grad_norm.py",
                                  "test_gpu_decoder_layer.py"])
def test_suite_under_the_debug_build(name):
    pact_build.build_debug()
    env = dict(os.environ, PACT_DEBUG="1")
    env["PYTHONPATH"] = os.pathsep.join(p for p in (ROOT, env.get("PYTHONPATH")) if p)
    # cases of tens of gigabytes are left to the release build
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-k", "not past_32_bits",
                        os.path.join(HERE, name)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
