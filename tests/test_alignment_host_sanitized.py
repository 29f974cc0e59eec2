"""The alignment operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU (the refusals of their C entry points)."""
import os
import subprocess
import sys

import pytest

from test_abi_host_sanitized import ROOT, san_env  # noqa: F401


@pytest.mark.parametrize("name", ["alignment", "logprobs", "int8"])
def test_refusals_pass_under_asan_and_ubsan(san_env, name):  # noqa: F811
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join("tests", f"test_{name}_validation.py")],
                       env=san_env, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=900)
    out = r.stdout.decode(errors="replace")
    assert r.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out
