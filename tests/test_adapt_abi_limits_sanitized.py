"""The edges of what the adapters' calls take against the build of the library whose host
code runs under AddressSanitizer and UndefinedBehaviorSanitizer, as test_adapt_abi_sanitized.py
does for the other argument checks."""
import os
import subprocess
import sys

import pytest

from sparse_gemm_layers_amd import build as B
from test_abi_sanitized import ROOT, _stale
from test_adapt_abi_sanitized import HEADERS

FILES = ["test_adapt_abi_limits.py", "test_adapt_plans.py"]


@pytest.mark.timeout(600)
def test_adapt_abi_limits_under_host_sanitizers():
    if os.environ.get("SG_LIBRARY"):
        pytest.skip("already running against another library build")
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    if _stale() or any(os.path.getmtime(h) > os.path.getmtime(B.SAN_LIB) for h in HEADERS):
        B.build(verbose=False, sanitize=True)
    env = dict(os.environ, LD_PRELOAD=B.host_sanitizer_runtime(), SG_LIBRARY=B.SAN_LIB,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-s", "-q", "-p", "no:cacheprovider",
                        *(os.path.join(ROOT, "tests", f) for f in FILES)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=500)
    out = r.stdout + r.stderr
    assert "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
