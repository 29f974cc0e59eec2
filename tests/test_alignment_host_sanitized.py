"""The alignment operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU (the refusals of their C entry points)."""
import os
import subprocess
import sys

from test_abi_host_sanitized import ROOT, san_env  # noqa: F401


def test_alignment_refusals_pass_under_asan_and_ubsan(san_env):  # noqa: F811
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join("tests", "test_alignment_validation.py")],
                       env=san_env, cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=900)
    out = r.stdout.decode(errors="replace")
    assert r.returncode == 0, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out
