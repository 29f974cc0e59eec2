"""The embedding's gradient beyond one sorting launch, against its fp64 definition: sorts of one to three passes by
small and large workgroups (up to and beyond 2^18 tokens), chunks of 32 to 128 tokens, runs that begin and end anywhere
in them.  Tolerances as derived in test_gpu_embedding.py."""
import numpy as np
import pytest

from test_gpu_embedding import grad_bound, zipf
from test_gpu_norm import np64

pytestmark = pytest.mark.gpu


def _check(flce_lib, ids, h, v, dtype, seed, accumulate=False, int32=False):
    import torch
    rng = np.random.default_rng(seed)
    g = torch.from_numpy(rng.normal(size=(len(ids), h))).to(getattr(torch, dtype))
    g[torch.from_numpy((ids < 0) | (ids >= v))] = float("nan")                 # never read
    base = torch.from_numpy(rng.normal(size=(v, h))).to(getattr(torch, dtype)) if accumulate else None
    on = torch.from_numpy(ids.astype(np.int32) if int32 else ids).cuda()
    got = flce_lib.embedding_backward(g.cuda(), on, v, scale=1.5, grad_weight=None if base is None else base.cuda())
    want, tol = grad_bound(ids, v, np64(g), 1.5, dtype, None if base is None else np64(base))
    err = np.abs(np64(got) - want)
    assert np.all(err <= tol), float(np.nanmax(err / tol))
    if accumulate:
        rest = np.ones(v, bool)
        rest[ids[(ids >= 0) & (ids < v)]] = False
        assert torch.equal(got.cpu()[torch.from_numpy(rest)], base[torch.from_numpy(rest)])


# 16384 | 16385: one launch and three a pass; 2^18 and one more: workgroups of 4 and of 16 waves.  V below 2^9, 2^18 and
# from there on: one, two and three passes, after which the sorted tokens stand in either buffer.
@pytest.mark.parametrize("v", [300, 511, 512, 5000, (1 << 18) - 1, 1 << 18, 300000])
@pytest.mark.parametrize("n", [16384, 16385, 20000, 1 << 18, (1 << 18) + 1, 300001])
def test_passes_and_workgroups(flce_lib, n, v):
    print(f"n={n} v={v}", flush=True)
    _check(flce_lib, zipf(np.random.default_rng(n + v), n, v), 8, v, "float32", seed=n)


@pytest.mark.parametrize("dtype,h", [("bfloat16", 8), ("bfloat16", 5), ("float16", 12), ("float32", 5)])
@pytest.mark.parametrize("n,v", [(20000, 300000), (300001, 5000)])
@pytest.mark.parametrize("accumulate,int32", [(False, True), (True, False)])
def test_types_and_buffers(flce_lib, n, v, dtype, h, accumulate, int32):
    print(f"n={n} v={v} h={h} {dtype}", flush=True)
    _check(flce_lib, zipf(np.random.default_rng(h), n, v), h, v, dtype, seed=h, accumulate=accumulate, int32=int32)


@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 200, 1000, 150001])
def test_ragged_runs_in_chunks_of_128(flce_lib, length):
    """Runs of about `length` tokens, so that their ends fall on every place of a chunk and of its 64-token rounds."""
    n = 300001
    rng = np.random.default_rng(length)
    print(f"length={length}", flush=True)
    lengths = np.maximum(1, length + rng.integers(-1, 2, size=n // length + 2))
    ids = np.repeat(np.arange(len(lengths)), lengths)[:n]
    v = int(ids.max()) + 1
    _check(flce_lib, rng.permutation(ids), 4, v, "float32", seed=length)
