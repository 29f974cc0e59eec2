"""layer_norm on the GPU against its fp64 definition.

Tolerances, before any run (u = 2^-24, half a step of fp32; e half a step of the output's type).  A sum of H terms
over 64 threads or more is a chain of at most H / 64 additions and a tree, so each sum is off by at most
K u of its absolute terms, K = H / 64 + 32 with the roundings of its terms.
 xhat = (x - mean) rstd is off by K u (|xhat| + rstd mean|x|) = K u X.
 y: e |y| + K u (|w| X + |b|).
 dx = rstd (d - s1 - xhat s2): e |dx| + K u rstd (|d| + mean|d| + X |s2| + |xhat| mean(|d| (|xhat| + X))), doubled
 for the products' own roundings.
 dweight: e |dw| + (K + N / 64 + 32) u sum |dy| (|xhat| + X);  dbias: e |db| + (K + N / 64 + 32) u sum |dy|.
1e-30 is added for underflow (fp16 outputs: their smallest step, 2^-25)."""
import numpy as np
import pytest

from oracle import ends_oracle as eo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 1e-30, "bfloat16": 1e-30, "float16": 2.0 ** -25}


def np64(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def problem(n, h, dtype, pdtype, seed=0, weight=True, bias=True, spread=1.0):
    import torch
    rng = np.random.default_rng(seed)
    dt, pt = getattr(torch, dtype), getattr(torch, pdtype)
    x = torch.from_numpy(rng.normal(size=(n, h)) * np.exp(0.5 * rng.normal(size=(n, 1))) + spread * rng.normal(size=(n, 1)))
    g = torch.from_numpy(rng.normal(size=(n, h)))
    w = torch.from_numpy(1 + 0.3 * rng.normal(size=h)).to(pt) if weight else None
    b = torch.from_numpy(0.3 * rng.normal(size=h)).to(pt) if bias else None
    return x.to(dt), w, b, g.to(dt)


def bounds(x, w, b, g, eps, dtype, pdtype):
    """Want and tolerance of y, dx, dw, db."""
    n, h = x.shape
    k = (h / 64 + 32) * U
    kn = k + (n / 64 + 32) * U
    y, xhat, rstd, _ = eo.layer_norm(x, w, b, eps)
    dx, dw, db = eo.layer_norm_grads(x, w, eps, g)
    one = np.ones(h) if w is None else w
    X = np.abs(xhat) + rstd * np.abs(x).mean(1, keepdims=True)
    d = np.abs(g * one)
    s2 = np.abs((g * one * xhat).mean(1, keepdims=True))
    e, ep, tiny, tinyp = HALF[dtype], HALF[pdtype], TINY[dtype], TINY[pdtype]
    ty = e * np.abs(y) + k * (np.abs(one) * X + (0 if b is None else np.abs(b))) + tiny
    tx = e * np.abs(dx) + 2 * k * rstd * (d + d.mean(1, keepdims=True) + X * s2
                                          + np.abs(xhat) * (d * (np.abs(xhat) + X)).mean(1, keepdims=True)) + tiny
    tw = ep * np.abs(dw) + kn * (np.abs(g) * (np.abs(xhat) + X)).sum(0) + tinyp
    tb = ep * np.abs(db) + kn * np.abs(g).sum(0) + tinyp
    return (y, ty), (dx, tx), (dw, tw), (db, tb)


def compare(got, want, tol, what):
    err = np.abs(np64(got) - want)
    assert np.all(err <= tol), (what, float((err / tol).max()))


def check(flce_lib, x, w, b, g, dtype, pdtype, eps=1e-5, on=None):
    import torch
    leaves = [None if t is None else t.cuda().requires_grad_(True) for t in (x, w, b)]
    y = flce_lib.layer_norm(*leaves, eps=eps)
    wanted = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad(y, wanted, g.cuda()))
    grads = [None if t is None else next(grads) for t in leaves]
    ref = bounds(np64(x), None if w is None else np64(w), None if b is None else np64(b), np64(g), eps, dtype, pdtype)
    assert y.dtype == x.dtype and y.is_contiguous()
    for t, leaf in zip(grads, leaves):
        assert t is None or (t.dtype == leaf.dtype and t.shape == leaf.shape)
    with torch.no_grad():
        assert torch.equal(flce_lib.layer_norm(*leaves, eps=eps), y)
    for name, t, (want, tol) in zip(("y", "dx", "dw", "db"), (y, *grads), ref):
        if t is not None:
            compare(t, want, tol, name)


SHAPES = [(1, 1), (3, 7), (5, 64), (16, 4096), (70, 1023), (33, 5000), (2, 16392), (700, 128), (300, 520), (9, 40000),
          (4, 8192), (1, 2048), (257, 1024), (6, 4104), (5, 16384), (3, 1 << 17), (66, 16385), (130, 17000)]


@pytest.mark.parametrize("dtype,pdtype", [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"),
                                          ("float16", "float16"), ("float16", "float32")])
@pytest.mark.parametrize("n,h", SHAPES)
def test_values_and_gradients(flce_lib, n, h, dtype, pdtype):
    check(flce_lib, *problem(n, h, dtype, pdtype, seed=n + h), dtype, pdtype)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("h", [72, 1001])
def test_without_weight_or_bias(flce_lib, h, weight, bias):
    check(flce_lib, *problem(37, h, "bfloat16", "float32", seed=h, weight=weight, bias=bias), "bfloat16", "float32",
          eps=1e-3)


@pytest.mark.parametrize("n,h", [(8192, 256), (5000, 97)])
def test_many_rows(flce_lib, n, h):
    check(flce_lib, *problem(n, h, "bfloat16", "float32", seed=5), "bfloat16", "float32")


@pytest.mark.parametrize("h,offset", [(512, 0), (512, 1), (500, 3)])
def test_rows_apart_and_unaligned(flce_lib, h, offset):
    """Slices of a wider tensor, x and the upstream gradient alike."""
    import torch
    x, w, b, g = problem(19, h, "float16", "float16", seed=h)
    wide = [torch.full((19, 2 * h + 8), float("nan"), dtype=t.dtype) for t in (x, g)]
    for t, into in zip((x, g), wide):
        into[:, offset:offset + h] = t
    xs, gs = (t.cuda()[:, offset:offset + h] for t in wide)
    leaves = [xs.requires_grad_(True), w.cuda().requires_grad_(True), b.cuda().requires_grad_(True)]
    y = flce_lib.layer_norm(*leaves)
    got = (y, *torch.autograd.grad(y, leaves, gs))
    for name, t, (want, tol) in zip(("y", "dx", "dw", "db"), got, bounds(np64(x), np64(w), np64(b), np64(g), 1e-5,
                                                                         "float16", "float16")):
        compare(t, want, tol, name)


def test_no_rows(flce_lib):
    import torch
    leaves = [torch.empty(0, 64, device="cuda", requires_grad=True), torch.ones(64, device="cuda", requires_grad=True),
              torch.zeros(64, device="cuda", requires_grad=True)]
    y = flce_lib.layer_norm(*leaves)
    gx, gw, gb = torch.autograd.grad(y, leaves, torch.empty(0, 64, device="cuda"))
    assert y.shape == gx.shape == (0, 64) and not gw.any() and not gb.any()


@pytest.mark.parametrize("h", [64, 1000, 4096, 20000])
def test_equal_values_and_infinities(flce_lib, h):
    """A row of equal values gives the bias (its mean is exact for a power of two); a row with an infinity or NaN
    gives NaN, and no other row is touched."""
    import torch
    x, w, b, _ = problem(6, h, "float32", "float32", seed=h)
    x[1] = 4.0
    x[2, h // 2] = float("inf")
    x[4, h - 1] = float("nan")
    y = flce_lib.layer_norm(x.cuda(), w.cuda(), b.cuda()).cpu()
    assert torch.equal(y[1], b) if h & (h - 1) == 0 else torch.allclose(y[1], b, atol=1e-2)
    assert y[2].isnan().all() and y[4].isnan().all()
    rest = [0, 3, 5]
    (want, tol), *_ = bounds(np64(x[rest]), np64(w), np64(b), np.zeros((3, h)), 1e-5, "float32", "float32")
    compare(y[rest], want, tol, "y")


@pytest.mark.parametrize("mean", [1e3, -3e4])
def test_far_from_zero(flce_lib, mean):
    """Rows whose mean is far larger than their spread: the tolerance grows with mean|x| / spread, no more."""
    import torch
    rng = np.random.default_rng(3)
    x = torch.from_numpy(mean + rng.normal(size=(8, 2048))).float()
    _, w, b, g = problem(8, 2048, "float32", "float32")
    check(flce_lib, x, w, b, g, "float32", "float32")


def test_only_some_gradients(flce_lib):
    import torch
    x, w, b, g = (t.cuda() for t in problem(40, 136, "bfloat16", "bfloat16"))
    full = [t.clone().requires_grad_(True) for t in (x, w, b)]
    want = torch.autograd.grad(flce_lib.layer_norm(*full), full, g)
    for k in range(3):
        leaves = [t.clone().requires_grad_(i == k) for i, t in enumerate((x, w, b))]
        got, = torch.autograd.grad(flce_lib.layer_norm(*leaves), leaves[k], g)
        assert torch.equal(got, want[k])


def test_expanded_upstream_gradient(flce_lib):
    """.sum() hands over one value for all places."""
    import torch
    x, w, b, _ = problem(12, 200, "float32", "float32")
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    flce_lib.layer_norm(*leaves).sum().backward()
    ref = bounds(np64(x), np64(w), np64(b), np.ones((12, 200)), 1e-5, "float32", "float32")
    for name, t, (want, tol) in zip(("dx", "dw", "db"), leaves, ref[1:]):
        compare(t.grad, want, tol, name)


def test_gradients_along_differences(flce_lib):
    """The kernels' gradients along a direction against central differences of the fp64 values (t = 1e-4: off by
    1e-8 of the sum of absolute terms, see test_norm_validation.py)."""
    import torch
    x, w, b, g = problem(20, 300, "float32", "float32", seed=9)
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    grads = torch.autograd.grad(flce_lib.layer_norm(*leaves), leaves, g.cuda())
    a = [np64(t) for t in (x, w, b)]
    ref = bounds(*a, np64(g), 1e-5, "float32", "float32")[1:]
    rng = np.random.default_rng(4)
    for k, grad in enumerate(grads):
        v = rng.normal(size=a[k].shape)
        v /= np.abs(v).max()

        def f(s):
            moved = list(a)
            moved[k] = a[k] + s * v
            return (np64(g) * eo.layer_norm(*moved, 1e-5)[0]).sum()

        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        tol = (ref[k][1] * np.abs(v)).sum() + 1e-6 * np.abs(np64(grad) * v).sum()
        assert abs(slope - (np64(grad) * v).sum()) <= tol


def test_no_second_derivative(flce_lib):
    """create_graph gives the same gradients; differentiating them is refused, not answered with zeros."""
    import torch
    x, w, b, g = (t.cuda() for t in problem(5, 40, "float32", "float32"))
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    want = torch.autograd.grad(flce_lib.layer_norm(*leaves), leaves, g)
    got = torch.autograd.grad(flce_lib.layer_norm(*leaves), leaves, g, create_graph=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(RuntimeError):
        got[0].sum().backward()


def test_backward_twice_and_retained(flce_lib):
    import torch
    x, w, b, g = (t.cuda() for t in problem(30, 64, "float32", "float32"))
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    y = flce_lib.layer_norm(*leaves)
    first = torch.autograd.grad(y, leaves, g, retain_graph=True)
    assert all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(y, leaves, g), first))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, leaves, g)
    y = flce_lib.layer_norm(*leaves)
    with torch.no_grad():
        x.add_(1)                                            # what the backward needs is gone
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, leaves, g)


def test_under_no_grad_and_inference_mode(flce_lib):
    import torch
    x, w, b, _ = (t.cuda() for t in problem(9, 72, "bfloat16", "float32"))
    want = flce_lib.layer_norm(x, w, b)
    x.requires_grad_(True)
    with torch.no_grad():
        assert torch.equal(flce_lib.layer_norm(x, w, b), want) and not flce_lib.layer_norm(x, w, b).requires_grad
    with torch.inference_mode():
        assert torch.equal(flce_lib.layer_norm(x, w, b), want)


def test_repeats_are_bitwise_equal_on_another_stream(flce_lib):
    import torch
    x, w, b, g = (t.cuda() for t in problem(1500, 512, "bfloat16", "float32"))
    leaves = [t.requires_grad_(True) for t in (x, w, b)]

    def step():
        y = flce_lib.layer_norm(*leaves)
        return (y, *torch.autograd.grad(y, leaves, g))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [step() for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_captured_step_replays(flce_lib):
    import torch
    x, w, b, g = (t.cuda() for t in problem(300, 256, "bfloat16", "bfloat16"))
    leaves = [t.requires_grad_(True) for t in (x, w, b)]

    def step():
        y = flce_lib.layer_norm(*leaves)
        return (y.detach(), *torch.autograd.grad(y, leaves, g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).to(x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, step()):
            assert torch.equal(p, q)


def test_beyond_32_bit_offsets(flce_lib):
    """More than 2^31 elements: the last rows are as a call of their own gives them."""
    import torch
    rows, h = (1 << 20) + 3, 2056
    x = torch.empty(rows, h, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.rand(h, device="cuda")
    y = flce_lib.layer_norm(x, w)
    assert torch.equal(y[-5:], flce_lib.layer_norm(x[-5:].clone(), w))
    assert torch.equal(y[:5], flce_lib.layer_norm(x[:5].clone(), w))
    xs = x[-5:].clone().requires_grad_(True)
    want, = torch.autograd.grad(flce_lib.layer_norm(xs, w), xs, x[-5:])
    x.requires_grad_(True)
    got, = torch.autograd.grad(flce_lib.layer_norm(x, w), x, x.detach())
    assert torch.equal(got[-5:], want)


@pytest.mark.parametrize("grad_mode", [True, False])
def test_dual_inputs_are_refused(flce_lib, grad_mode):
    import torch
    import torch.autograd.forward_ad as fwAD
    x, w, b, _ = (t.cuda() for t in problem(3, 16, "float32", "float32"))
    with torch.set_grad_enabled(grad_mode), fwAD.dual_level():
        for k in range(3):
            a = [x, w, b]
            a[k] = fwAD.make_dual(a[k], torch.ones_like(a[k]))
            with pytest.raises(NotImplementedError):
                flce_lib.layer_norm(*a)
