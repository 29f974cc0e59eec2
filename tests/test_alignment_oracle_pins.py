"""The alignment oracle against closed forms and against differences (CPU)."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao


def _difference(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += eps
        down[i] -= eps
        g[i] = (f(up) - f(down)) / (2 * eps)
    return g


def test_logprobs_of_a_uniform_head_and_of_a_certain_one():
    x, w = np.ones((2, 4)), np.zeros((5, 4))
    logp, ent, _, _ = ao.token_logprobs(x, w, None, np.array([3, -100]))
    assert np.allclose(logp, [-np.log(5), 0]) and np.allclose(ent, [np.log(5), 0])
    b = np.array([0.0, -np.inf, -np.inf, -np.inf, -np.inf])
    logp, ent, _, _ = ao.token_logprobs(x, w, b, np.array([0, 1]))
    assert np.array_equal(logp, [0, -np.inf]) and np.array_equal(ent, [0, 0])


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_logprob_gradients_against_differences(cap):
    rng = np.random.default_rng(0)
    x, w, b = rng.normal(size=(3, 4)), rng.normal(size=(6, 4)), rng.normal(size=6)
    t, g, h = np.array([2, -100, 5]), rng.normal(size=3), rng.normal(size=3)
    opts = dict(logit_scale=0.7, softcap=cap)

    def value(x_, w_, b_):
        logp, ent, _, _ = ao.token_logprobs(x_, w_, b_, t, **opts)
        return g @ logp + h @ ent

    gx, gw, gb = ao.token_logprobs_grads(x, w, b, t, g, h, **opts)
    assert np.allclose(gx, _difference(lambda v: value(v, w, b), x), atol=1e-8)
    assert np.allclose(gw, _difference(lambda v: value(x, v, b), w), atol=1e-8)
    assert np.allclose(gb, _difference(lambda v: value(x, w, v), b), atol=1e-8)


def test_quantize_rows():
    q, s = ao.quantize_int8(np.array([[1.0, -127.0, 63.5], [0, 0, 0], [np.inf, 1, 1], [1e-40, 0, 0]], np.float32))
    assert q.tolist() == [[1, -127, 64], [0, 0, 0], [0, 0, 0], [0, 0, 0]]
    assert s[0] == 1.0 and s[1] == 0.0 and np.isnan(s[2]) and s[3] == 0.0


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("normalize", [False, True])
def test_preference_gradient_against_differences(kind, normalize):
    rng = np.random.default_rng(1)
    lp, ref = rng.normal(size=(6, 5)), rng.normal(size=(6, 5))
    mask = rng.random((6, 5)) < 0.7
    mask[4] = False
    g = rng.normal(size=3)
    opts = dict(beta=0.3, loss_type=kind, margin=0.2, length_normalize=normalize, reduction="none",
                label_smoothing=0.1 if kind == "sigmoid" else 0.0)
    _, _, grad = ao.preference(lp, ref, None, mask, **opts)
    want = _difference(lambda v: g @ ao.preference(v, ref, None, mask, **opts)[0], lp)
    assert np.allclose(grad(g), want, atol=1e-7)


def test_preference_closed_form():
    # one pair, one token each: h = beta (1 - (-1)) = 1
    loss, rewards, _ = ao.preference(np.array([[1.0], [-1.0]]), None, beta=0.5)
    assert np.isclose(loss, np.log1p(np.exp(-1.0))) and np.allclose(rewards, [0.5, -0.5])


@pytest.mark.parametrize("reduction", ["none", "sum", "mean", "sequence_mean"])
@pytest.mark.parametrize("packed", [False, True])
def test_policy_gradient_against_differences(reduction, packed):
    rng = np.random.default_rng(2)
    shape = (20,) if packed else (4, 5)
    off = np.array([0, 7, 7, 16, 19]) if packed else None
    lp = rng.normal(size=shape)
    old, ref, ent = lp + rng.normal(size=shape), lp + rng.normal(size=shape), rng.random(shape)
    adv, mask = rng.normal(size=4), rng.random(shape) < 0.8
    g = rng.normal(size=shape if reduction == "none" else ())
    opts = dict(dual_clip=2.0, kl_coef=0.3, entropy_coef=0.2, reduction=reduction)
    out = ao.policy(lp, old, adv, ref, ent, off, mask, **opts)
    f = lambda a, b: np.sum(g * ao.policy(a, old, adv, ref, b, off, mask, **opts)["loss"])  # noqa: E731
    assert np.allclose(out["grad"](g), _difference(lambda v: f(v, ent), lp), atol=1e-7)
    assert np.allclose(out["grad_entropy"](g), _difference(lambda v: f(lp, v), ent), atol=1e-7)


def test_policy_closed_form():
    # ratios 2, 1/2, 2, 1/2 with advantages 1, 1, -1, -1 at clip 0.2: 1.2, 0.5, -2, -0.8
    lp, old = np.log([[2.0, 0.5, 2.0, 0.5]]), np.zeros((1, 4))
    out = ao.policy(lp, old, np.array([[1.0, 1.0, -1.0, -1.0]]), reduction="none")
    assert np.allclose(out["loss"], [[-1.2, -0.5, 2.0, 0.8]])
    assert np.allclose(out["grad"](1.0), [[0, -0.5, 2.0, 0]]) and out["clip_fraction"] == 0.5
