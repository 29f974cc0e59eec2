"""token_logprobs' gradients against differences of its own values, along directions in which the derivative
is as large as it can be, log-probabilities and entropies each for itself.

Tolerances, before any run: the values' bound of test_gpu_token_logprobs.py, summed over the rows that
count with their weights and divided by the step, and the difference's truncation, which is 4/3 of what halving the
step changes in fp64 for a smooth function (taken twice); the gradients' own fp32 rounding is far below both.
The step is the one, of powers of two, for which that sum is least: it is found from the fp64 values alone."""
import math

import pytest

from test_gpu_token_logprobs import U32, _tensors

pytestmark = pytest.mark.gpu
CAP, SCALE, ROWS = 6.0, 0.8, 60


def _values64(x, w, b, t):
    """(logp, entropy, z, the logits' terms) in fp64."""
    import torch
    z = CAP * torch.tanh(SCALE * (x @ w.t().contiguous() + b) / CAP)
    lp = z - torch.logsumexp(z, 1, keepdim=True)
    at = t.clamp_min(0)[:, None]
    return lp.gather(1, at)[:, 0], -(lp.exp() * lp).sum(1), z, (x.abs() @ w.abs().t().contiguous() + b.abs()).amax(1)


# both sides of the choice between small and large tiles, up to and above 64 tokens
@pytest.mark.parametrize("n,h,v", [(60, 64, 300), (200, 64, 1000), (2048, 64, 16384)])
@pytest.mark.parametrize("which", ["logps", "entropy"])
def test_gradients_match_differences(flce_lib, n, h, v, which):
    import torch
    x, w, b, t = _tensors(n, h, v, "f32", seed=11)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w, b)]
    t = t.cuda()
    gen = torch.Generator().manual_seed(3)
    g = torch.zeros(n)
    rows = torch.randperm(n, generator=gen)[:ROWS]
    g[rows] = torch.randn(rows.numel(), generator=gen)
    g = torch.where(t.cpu() >= 0, g, 0.0).cuda()

    def values(a):
        lp, ent = flce_lib.token_logprobs(a[0], a[1], t, a[2], logit_scale=SCALE, softcap=CAP, return_entropy=True)
        return lp if which == "logps" else ent

    def f(a):
        with torch.no_grad():
            return (g.double() * values(a).double()).sum().item()

    def f64(a):
        out = _values64(*a, t)
        return (g.double() * (out[0] if which == "logps" else out[1])).sum().item()

    grads = torch.autograd.grad(values(leaves), leaves, g)

    def rounding(a):
        _, _, z, terms = _values64(*(x.double() for x in a), t)
        ez = SCALE * terms * U32 * (h + 8) + 3 * U32 * CAP
        own = 8 * U32 * (z.abs().amax(1) + math.log(v) + 1)
        spread = 1 + 2 * (z.amax(1) - z.amin(1) + math.log(v))
        return (g.double().abs() * (2 * ez + own if which == "logps" else spread * ez + 2 * own)).sum().item()

    for k, name in enumerate(("hidden", "weight", "bias")):
        d = grads[k] / grads[k].norm()
        noise = torch.randn(d.shape, generator=torch.Generator().manual_seed(k)).cuda()
        d = d + 0.3 * noise / noise.norm()

        def moved(s):
            return [(a.detach() + (s * d if i == k else 0)) for i, a in enumerate(leaves)]

        def difference(fn, s, cast):
            up, down = ([cast(a) for a in moved(q)] for q in (s, -s))
            return (fn(up) - fn(down)) / (2 * s)

        def tolerance(s):
            halved = difference(f64, s, lambda a: a.double()) - difference(f64, s / 2, lambda a: a.double())
            return (rounding(moved(s)) + rounding(moved(-s))) / (2 * s) + 2 * 4 / 3 * abs(halved)

        tol, eps = min((tolerance(2.0 ** e), 2.0 ** e) for e in range(-4, 4))
        # the moved leaves are rounded to fp32: the derivative along what was really moved
        real = (moved(eps)[k].double() - moved(-eps)[k].double()) / (2 * eps)
        want = (grads[k].double() * real).sum().item()
        diff = difference(f, eps, lambda a: a)
        assert tol <= 0.25 * abs(want), (name, eps, tol, want)        # the test says something
        assert abs(diff - want) <= tol, (name, eps, diff, want, tol)
