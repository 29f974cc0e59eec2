"""Every launch of an entry point that fails is reported by that call, whichever of its launches it is: on the CPU, in a
child process whose launches go to a stand-in runtime that refuses one of them and, as HIP does, hands out its error
once."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = r"""
static int fail_at, count, last;   /* fail_at: number of the launch that is refused, from 1; 0 = none */
void stand_in_reset(int k) { fail_at = k; count = last = 0; }
int stand_in_count(void) { return count; }
int hipLaunchKernel(void) {
  if (++count == fail_at) return last = 9;   /* hipErrorInvalidConfiguration */
  return 0;
}
int hipGetLastError(void) { const int e = last; last = 0; return e; }
int hipPeekAtLastError(void) { return last; }
int __hipPushCallConfiguration(void) { return 0; }
int __hipPopCallConfiguration(void) { return 0; }
"""

CHILD = r"""
import ctypes, sys
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import linear_cross_entropy_tiled_amd as f
P, BIG = 4096, 1 << 40      # an aligned address that is never followed, and room for any workspace

def scores(n, h, v, codes):
    p = f.make_params(n, h, v, reduction="none")
    return lambda: f.flce_logprobs_mxfp4(p, P, P if codes else None, P, P, None, P, P, P, P, P, BIG, None)

def norm(cols, back):
    p = f.flce_norm_params(100, cols, 0, 0, f.DTYPES["bf16"], f.DTYPES["f32"], 1e-5, 0)
    if back:
        return lambda: f.flce_layer_norm_backward(p, P, P, P, P, P, P, P, P, P, BIG, None)
    return lambda: f.flce_layer_norm_forward(p, P, P, P, P, P, P, None)

def embedding(n, back, address=P):
    p = f.flce_embedding_params(n, 64, 1000, -100, f.DTYPES["bf16"], f.DTYPES["bf16"], 0, 1.0)
    if back:
        return lambda: f.flce_embedding_backward(p, P, P, address, P, BIG, None)
    return lambda: f.flce_embedding_forward(p, P, P, P, None)

def logprobs(int8):
    p = f.make_params(300, 256, 5000, reduction="none")
    if int8:
        return lambda: f.flce_logprobs_int8(p, P, P, P, P, None, P, P, P, P, P, BIG, None)
    return lambda: f.flce_logprobs_forward(p, P, P, None, P, P, P, P, P, BIG, None)

calls = {f"scores of {n} x {h} x {v}, {'codes' if c else 'values'}": scores(n, h, v, c)
         for n, h, v in ((4, 64, 300), (4, 128, 300), (1000, 2048, 50001), (1000, 2080, 50001), (0, 64, 300))
         for c in (False, True)}
calls.update({f"norm of {cols}, {'backward' if b else 'forward'}": norm(cols, b)
              for cols in (64, 20000) for b in (False, True)})
calls.update({f"embedding of {n}, {'backward' if b else 'forward'}": embedding(n, b)
              for n in (50, 20000, 300000) for b in (False, True)})
calls["embedding of 50, backward into an odd address"] = embedding(50, True, P + 2)
calls["quantize"] = lambda: f.flce_quantize_mxfp4(1, P, 8, 64, P, P, None)
calls["dequantize"] = lambda: f.flce_dequantize_mxfp4(1, P, P, 8, 64, P, None)
calls["8-bit scores"] = logprobs(True)
calls["log-probabilities"] = logprobs(False)

for name, call in calls.items():
    stand_in.stand_in_reset(0)
    assert call() == f.FLCE_OK, name
    launches = stand_in.stand_in_count()
    assert launches > 0, name
    lost = []
    for k in range(1, launches + 1):
        stand_in.stand_in_reset(k)
        if call() != f.FLCE_ERR_HIP:
            lost.append(k)
    print(f"{name}: {launches} launches" + (f", LOST {lost}" if lost else ""), flush=True)
"""


def test_a_launch_that_fails_is_reported(tmp_path):
    cc = shutil.which("cc") or shutil.which("gcc") or shutil.which("clang")
    if cc is None:
        pytest.skip("no C compiler")
    import linear_cross_entropy_tiled_amd as flce
    if not os.path.exists(flce.LIB_PATH):
        pytest.skip("libflce.so is not built")
    src, lib = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       timeout=300)
    out = r.stdout.decode(errors="replace")
    assert r.returncode == 0, out[-3000:]
    assert out.count("launches") >= 20 and "LOST" not in out, out
