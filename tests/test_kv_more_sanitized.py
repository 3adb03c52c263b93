"""The refusals of forms, compaction and pool (test_kv_more_host.py) under AddressSanitizer and UndefinedBehaviorSanitizer (CPU), in the
sanitized copy of the host layer that test_capi_sanitized.py describes."""
import os
import subprocess
import sys

import pytest

from tests.test_capi_sanitized import ROOT, _asan_runtime


def test_kv_more_host_validation_under_sanitizers():
    rt = _asan_runtime()
    if rt is None or not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("no hipcc or clang sanitizer runtime in this environment")
    from sparse_kv_retrieval_amd import build as B
    pkg_parent = os.path.dirname(B.build_sanitized_host())
    env = dict(os.environ, PYTHONPATH=pkg_parent, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not binding",
                        "--import-mode=append", "--rootdir", ROOT, os.path.join(ROOT, "tests", "test_kv_more_host.py")],
                       cwd=pkg_parent, env=env, capture_output=True, text=True, timeout=600)
    report = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, report + "\nRC=" + str(r.returncode)
    assert "AddressSanitizer" not in report and "runtime error:" not in report, report
