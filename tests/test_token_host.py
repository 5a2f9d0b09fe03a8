"""The token-side operators' validation and plans under the host sanitizers.

``kan_token_api.cpp`` is compiled for the host only with AddressSanitizer and
UndefinedBehaviorSanitizer (the first report aborts) and linked against the
stubs and the walk over shapes of ``host/token_driver.cpp``.
"""

import os
import subprocess

import pytest

from test_host_sanitize import CSRC, HERE, ROOT, _hipcc


def test_plans_and_validation_under_sanitizers(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "token_driver")
    cmd = [cc, "--offload-host-only", "-std=c++17", "-O1", "-g",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-fno-sanitize-recover=all", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o", out,
           os.path.join(CSRC, "kan_token_api.cpp"), os.path.join(HERE, "host", "token_driver.cpp")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([out], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0 and "Sanitizer" not in res.stderr and "runtime error" not in res.stderr, \
        res.stderr[-4000:]
    assert res.stdout.startswith("ok ")
