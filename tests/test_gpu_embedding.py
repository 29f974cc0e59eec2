"""embedding and its gradient on the GPU against their fp64 definitions.

Tolerances, before any run (u = 2^-24, e half a step of the output's type).  Forward: scale is rounded to fp32, the
product too, then the output: (e + 2 u) |y|; a scale of 1 is exact.  Gradient: a run of c tokens is summed in
pieces, a chain of at most c additions, and never more than 64 + N / 2048 + c / 32; with the scale's, the product's
and (accumulated) the last addition's rounding: e |dw| + (chain + 4) u (scale sum |g| + |what was there|).
1e-30 is added for underflow (fp16 outputs: half their smallest step, 2^-25)."""
import numpy as np
import pytest

from oracle import ends_oracle as eo
from test_gpu_norm import HALF, TINY, U, np64

pytestmark = pytest.mark.gpu


def zipf(rng, n, v, ignored=0.05):
    """Frequent tokens, rare ones, some that are ignored, some that are no row."""
    ids = np.minimum(np.exp(rng.random(n) * np.log(v + 1)).astype(np.int64) - 1, v - 1)
    ids[rng.random(n) < ignored] = -100
    if n > 8:
        ids[rng.integers(0, n, 3)] = [v, -1, v + 12345]
    return ids


def problem(n, h, v, dtype, seed, ids=None):
    import torch
    rng = np.random.default_rng(seed)
    ids = zipf(rng, n, v) if ids is None else ids
    dt = getattr(torch, dtype)
    w = torch.from_numpy(rng.normal(size=(v, h))).to(dt)
    g = torch.from_numpy(rng.normal(size=(n, h))).to(dt)
    bad = (ids < 0) | (ids >= v)
    g[torch.from_numpy(bad)] = float("nan")                 # never read
    return torch.from_numpy(ids), w, g


def grad_bound(ids, v, g, scale, gdtype, base=None):
    n = len(ids)
    want, terms, count = eo.embedding_grad(ids, v, g, scale)
    chain = np.minimum(count, 64 + n / 2048 + count / 32)[:, None] + 4
    if base is not None:
        want, terms = want + base, terms + np.abs(base)
    return want, HALF[gdtype] * np.abs(want) + chain * U * terms + TINY[gdtype]


def check(flce_lib, ids, w, g, dtype, scale=1.0):
    import torch
    leaf = w.cuda().requires_grad_(True)
    y = flce_lib.embedding(ids.cuda(), leaf, scale=scale)
    want = eo.embedding(ids.numpy(), np64(w), scale)
    assert y.dtype == w.dtype and tuple(y.shape) == want.shape
    if scale == 1.0:
        assert np.array_equal(np64(y), want)
    else:
        assert np.all(np.abs(np64(y) - want) <= (HALF[dtype] + 2 * U) * np.abs(want) + TINY[dtype])
    grad, = torch.autograd.grad(y, leaf, g.cuda())
    want, tol = grad_bound(ids.numpy(), len(w), np64(g), scale, dtype)
    err = np.abs(np64(grad) - want)
    assert grad.dtype == w.dtype and np.all(err <= tol), float(np.nanmax(err / tol))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,h,v", [(1, 8, 1), (1, 1, 3), (7, 33, 5), (64, 512, 300), (500, 4096, 1000), (2001, 1023, 8191),
                                   (8192, 72, 500), (8193, 64, 70000), (3000, 2056, 300), (40000, 24, 131)])
def test_values_and_gradients(flce_lib, n, h, v, dtype):
    check(flce_lib, *problem(n, h, v, dtype, seed=n + h), dtype, scale=1.0 if n % 2 else 22.627417)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 1000, 8192, 9000, 200000])
@pytest.mark.parametrize("which", ["same", "distinct", "none", "pairs"])
def test_runs(flce_lib, n, which):
    """One run over everything, none longer than a token, no token at all, runs over every chunk's edge."""
    v = max(n, 4)
    ids = {"same": np.full(n, 3), "distinct": np.random.default_rng(n).permutation(n), "none": np.full(n, -100),
           "pairs": (np.arange(n) + 1) // 2 % v}[which].astype(np.int64)
    check(flce_lib, *problem(n, 16, v, "bfloat16", seed=n, ids=ids), "bfloat16")


@pytest.mark.parametrize("dtype,gdtype", [("bfloat16", "float32"), ("float32", "bfloat16"), ("float16", "float16"),
                                          ("float32", "float32")])
@pytest.mark.parametrize("h", [40, 41])
def test_added_to_what_is_there(flce_lib, h, dtype, gdtype):
    """embedding_backward into a tied head's buffer: the rows that do not occur keep their bits."""
    import torch
    n, v = 900, 700
    ids, _, g = problem(n, h, v, dtype, seed=h)
    base = torch.randn(v, h, generator=torch.Generator().manual_seed(1)).to(getattr(torch, gdtype))
    buf = base.cuda()
    out = flce_lib.embedding_backward(g.cuda(), ids.cuda(), v, scale=0.7, grad_weight=buf)
    assert out is buf
    want, tol = grad_bound(ids.numpy(), v, np64(g), 0.7, gdtype, np64(base))
    assert np.all(np.abs(np64(buf) - want) <= tol)
    untouched = np.ones(v, bool)
    untouched[ids.numpy()[(ids.numpy() >= 0) & (ids.numpy() < v)]] = False
    assert untouched.any() and torch.equal(buf.cpu()[untouched], base[untouched])
    fresh = flce_lib.embedding_backward(g.cuda(), ids.cuda(), v, scale=0.7,
                                        grad_weight_dtype={"float32": "f32", "bfloat16": "bf16", "float16": "f16"}[gdtype])
    want, tol = grad_bound(ids.numpy(), v, np64(g), 0.7, gdtype)
    assert fresh.dtype == base.dtype and np.all(np.abs(np64(fresh) - want) <= tol)


@pytest.mark.parametrize("first,rows", [(0, 100), (37, 63), (90, 10)])
def test_vocabulary_slices(flce_lib, first, rows):
    """Slices, at rows that are not 16-byte aligned, add up to the whole."""
    import torch
    ids, w, g = problem(300, 19, 100, "float32", seed=first)
    ids, w, g = ids.cuda(), w.cuda(), g.cuda()
    whole, part = flce_lib.embedding(ids, w), flce_lib.embedding(ids - first, w[first:first + rows], ignore_index=-100 - first)
    mine = ((ids >= first) & (ids < first + rows))[:, None]
    assert torch.equal(part, torch.where(mine, whole, 0.0))
    buf = torch.full((101, 19), 5.0, device="cuda")
    flce_lib.embedding_backward(g, ids - first, rows, ignore_index=-100 - first, grad_weight=buf[first:first + rows].zero_())
    want, tol = grad_bound(ids.cpu().numpy(), 100, np64(g), 1.0, "float32")
    assert np.all(np.abs(np64(buf[first:first + rows]) - want[first:first + rows]) <= tol[first:first + rows])
    assert (buf[:first] == 5).all() and (buf[first + rows:] == 5).all()


def test_int32_ids_and_ignore_index(flce_lib):
    import torch
    ids, w, g = problem(400, 32, 90, "bfloat16", seed=2)
    a = flce_lib.embedding(ids.cuda(), w.cuda())
    assert torch.equal(flce_lib.embedding(ids.int().cuda(), w.cuda()), a)
    assert torch.equal(flce_lib.embedding_backward(g.cuda(), ids.int().cuda(), 90),
                       flce_lib.embedding_backward(g.cuda(), ids.cuda(), 90))
    off = flce_lib.embedding(ids.cuda(), w.cuda(), ignore_index=5)          # a row of the weight, left out
    assert torch.equal(off, torch.where((ids == 5)[:, None].cuda(), 0.0, a.float()).to(a.dtype))
    g = torch.nan_to_num(g).cuda()
    assert not flce_lib.embedding_backward(g, ids.cuda(), 90, ignore_index=5)[5].any()


def test_no_tokens(flce_lib):
    import torch
    w = torch.ones(9, 16, device="cuda", requires_grad=True)
    y = flce_lib.embedding(torch.empty(0, dtype=torch.int64, device="cuda"), w)
    grad, = torch.autograd.grad(y, w, torch.empty(0, 16, device="cuda"))
    assert y.shape == (0, 16) and not grad.any()
    buf = torch.full((9, 16), 3.0, device="cuda")
    flce_lib.embedding_backward(y.detach(), torch.empty(0, dtype=torch.int64, device="cuda"), 9, grad_weight=buf)
    assert (buf == 3).all()


def test_infinities_stay_in_their_rows(flce_lib):
    import torch
    ids = torch.tensor([1, 2, 1, 4, 2], device="cuda")
    g = torch.ones(5, 8, device="cuda")
    g[1, 3], g[2, 0] = float("inf"), float("nan")
    grad = flce_lib.embedding_backward(g, ids, 6)
    assert grad[2, 3].isinf() and grad[1, 0].isnan()
    assert grad.isfinite().sum() == grad.numel() - 2


def test_gradient_along_differences(flce_lib):
    """The map is linear in weight: the difference of its fp64 values along a direction is the slope itself."""
    import torch
    ids, w, g = problem(700, 24, 130, "float32", seed=4)
    g = torch.nan_to_num(g)
    grad = np64(flce_lib.embedding_backward(g.cuda(), ids.cuda(), 130, scale=1.7))
    v = np.random.default_rng(1).normal(size=grad.shape)
    slope = (np64(g) * (eo.embedding(ids.numpy(), np64(w) + v, 1.7) - eo.embedding(ids.numpy(), np64(w) - v, 1.7))).sum() / 2
    _, tol = grad_bound(ids.numpy(), 130, np64(g), 1.7, "float32")
    assert abs(slope - (grad * v).sum()) <= (tol * np.abs(v)).sum() + 1e-9 * np.abs(grad * v).sum()


def test_no_second_derivative(flce_lib):
    import torch
    ids, w, g = problem(30, 8, 12, "float32", seed=3)
    ids, w, g = ids.cuda(), w.cuda().requires_grad_(True), torch.nan_to_num(g).cuda().requires_grad_(True)
    want, = torch.autograd.grad(flce_lib.embedding(ids, w), w, g)
    got, = torch.autograd.grad(flce_lib.embedding(ids, w), w, g, create_graph=True)
    assert torch.equal(got, want)
    with pytest.raises(RuntimeError):
        got.sum().backward()
    with torch.no_grad():
        assert not flce_lib.embedding(ids, w).requires_grad


def test_non_contiguous_upstream_gradient(flce_lib):
    import torch
    ids, w, _ = problem(50, 24, 30, "float32", seed=6)
    leaf = w.cuda().requires_grad_(True)
    flce_lib.embedding(ids.cuda(), leaf).sum().backward()
    want, tol = grad_bound(ids.numpy(), 30, np.ones((50, 24)), 1.0, "float32")
    assert np.all(np.abs(np64(leaf.grad) - want) <= tol)


def test_repeats_are_bitwise_equal_on_another_stream(flce_lib):
    import torch
    ids, w, g = problem(20000, 64, 500, "bfloat16", seed=7)
    ids, g = ids.cuda(), g.cuda()
    want = flce_lib.embedding_backward(g, ids, 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [flce_lib.embedding_backward(g, ids, 500) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("n", [700, 9000])
def test_captured_step_replays(flce_lib, n):
    import torch
    ids, w, g = problem(n, 64, 300, "bfloat16", seed=8)
    ids, w, g = ids.cuda(), w.cuda().requires_grad_(True), torch.nan_to_num(g).cuda()

    def step():
        y = flce_lib.embedding(ids, w)
        return y.detach(), *torch.autograd.grad(y, w, g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        ids.copy_(torch.from_numpy(zipf(np.random.default_rng(k), n, 300)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_beyond_32_bit_offsets(flce_lib):
    """Weights and outputs of more than 2^31 elements."""
    import torch
    v, h = (1 << 19) + 5, 4104
    w = torch.zeros(v, h, dtype=torch.bfloat16, device="cuda")
    w[-3:] = torch.arange(3, dtype=torch.bfloat16, device="cuda")[:, None] + 1
    ids = torch.tensor([v - 1, 0, v - 3, v], device="cuda")
    assert flce_lib.embedding(ids, w)[:, h - 1].tolist() == [3.0, 0.0, 1.0, 0.0]
    g = torch.ones(4, h, dtype=torch.bfloat16, device="cuda")
    out = flce_lib.embedding_backward(g, ids, v, grad_weight=w)
    assert out[-3:, h - 1].tolist() == [2.0, 2.0, 4.0] and out[0, 0] == 1 and not out[1:-3].any()
    del w, out
    many = torch.arange(3, device="cuda").repeat((1 << 20) // 2)            # outputs of 2^20 * 1.5 * 2056
    small = torch.arange(3 * 2056, device="cuda").view(3, 2056).to(torch.bfloat16)
    y = flce_lib.embedding(many, small)
    assert torch.equal(y[-3:], small) and torch.equal(y[:3], small)
    grad = flce_lib.embedding_backward(y, many, 3, grad_weight_dtype="f32")
    want = (many.numel() // 3) * small.double()
    assert ((grad.double() - want).abs() <= (64 + many.numel() / 2048 + many.numel() / 32) * U * want).all()


@pytest.mark.parametrize("grad_mode", [True, False])
def test_dual_inputs_are_refused(flce_lib, grad_mode):
    import torch
    import torch.autograd.forward_ad as fwAD
    w = torch.ones(4, 8, device="cuda")
    with torch.set_grad_enabled(grad_mode), fwAD.dual_level(), pytest.raises(NotImplementedError):
        flce_lib.embedding(torch.zeros(2, dtype=torch.int64, device="cuda"), fwAD.make_dual(w, torch.ones_like(w)))
