"""The argument checks of the routing and 4-bit entry points against the build of
the library whose host code runs under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitized.py does for the rest."""
import os
import subprocess
import sys

import pytest

from sparse_gemm_layers_amd import build as B
from test_abi_sanitized import ROOT, _stale

HEADER = os.path.join(B.HERE, "include", "sg_moe.h")


@pytest.mark.timeout(600)
def test_moe_abi_under_host_sanitizers():
    if os.environ.get("SG_LIBRARY"):
        pytest.skip("already running against another library build")
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    if _stale() or os.path.getmtime(HEADER) > os.path.getmtime(B.SAN_LIB):
        B.build(verbose=False, sanitize=True)
    runtime = B.host_sanitizer_runtime()
    assert os.path.exists(runtime), runtime
    env = dict(os.environ, LD_PRELOAD=runtime, SG_LIBRARY=B.SAN_LIB,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-s", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_moe_abi.py"),
                        os.path.join(ROOT, "tests", "test_moe_abi_limits.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=500)
    out = r.stdout + r.stderr
    assert "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
