"""token_logprobs on the GPU against the fp64 oracle: values, gradients, masks.

Tolerances, before any run.  Logits are fp32 sums of H products of exact 16-bit (or
rounded fp32) values: |error| <= (H / 32 + 8) x 2^-24 x sum |x w| per logit for the
16-bit matrix instructions' chain of H / 32 accumulations (fp32: H products and
additions, H + 8), with the bias and the scale.  A softcap adds its formula's
3 x 2^-24 cap.  log p and H move by at most twice resp. (1 + 2 |log p|) times the
logits' error, plus 8 x 2^-24 of the values' own size (lse <= |z| + ln V).
Gradients: the logit gradient is held in the input's type (one rounding, eps / 2 of
each entry), the outputs are rounded once more, and sums accumulate in fp32."""
import numpy as np
import pytest

import synth_inputs as si
from oracle import alignment_oracle as ao

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _tensors(n, h, v, dtype, seed, bias=True, ignored=0.1, weight_std=0.1):
    import torch
    rng = np.random.default_rng(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    x = torch.from_numpy(rng.normal(size=(n, h))).to(dt)
    w = torch.from_numpy(rng.normal(size=(v, h)) * weight_std).to(dt)
    b = torch.from_numpy(rng.normal(size=v) * 0.3).to(dt) if bias else None
    t = rng.integers(0, v, size=n)
    t[rng.random(n) < ignored] = -100
    return x, w, b, torch.from_numpy(t)


def _np(t):
    import torch
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def _bounds(x, w, b, dtype, opts):
    """Error bound of a row's logits (the worst of the row)."""
    h = x.shape[1]
    terms = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))
    z = np.abs(opts.get("logit_scale", 1.0)) * terms.max(axis=1) * U32 * ((h if dtype == "f32" else h / 32) + 8)
    return z + 3 * U32 * opts.get("softcap", 0.0)


def _check_values(logps, entropy, x, w, b, t, dtype, opts):
    want_lp, want_h, z, _ = ao.token_logprobs(x, w, b, t, softcap=opts.get("softcap") or 0.0,
                                              logit_scale=opts.get("logit_scale", 1.0))
    valid = (t >= 0) & (t < w.shape[0])
    assert not np.any(logps[~valid]) and not np.any(entropy[~valid])
    ez = _bounds(x, w, b, dtype, dict(opts, softcap=opts.get("softcap") or 0.0))
    own = 8 * U32 * (np.abs(z).max(axis=1) + np.log(w.shape[0]) + 1)
    assert np.all(np.abs(logps - want_lp)[valid] <= (2 * ez + own)[valid])
    spread = 1 + 2 * (z.max(axis=1) - z.min(axis=1) + np.log(w.shape[0]))
    assert np.all(np.abs(entropy - want_h)[valid] <= (spread * ez + 2 * own)[valid])
    return want_h


SHAPES = [(1, 8, 1), (1, 64, 1000), (3, 72, 257), (17, 136, 255), (255, 64, 513), (256, 128, 512), (300, 264, 2049),
          (515, 64, 5001), (1030, 40, 1100)]
OPTS = [dict(), dict(logit_scale=0.7, softcap=5.0)]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k", [0, 1])
def test_values_and_gradients(flce_lib, n, h, v, dtype, k):
    import torch
    opts = OPTS[k]
    x, w, b, t = _tensors(n, h, v, dtype, seed=n + h + v, bias=(n + k) % 2 == 0)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w, b) if a is not None]
    tt = (t.int() if k else t).cuda()
    lp, ent = flce_lib.token_logprobs(leaves[0], leaves[1], tt, leaves[2] if b is not None else None,
                                      return_entropy=True, vocab_chunk=512 if k else 0, **opts)
    X, W, B, T = _np(x), _np(w), _np(b), t.numpy()
    _check_values(_np(lp), _np(ent), X, W, B, T, dtype, opts)
    rng = np.random.default_rng(n)
    g, e = rng.normal(size=n).astype(np.float32), rng.normal(size=n).astype(np.float32)
    got = torch.autograd.grad((lp, ent), leaves, (torch.from_numpy(g).cuda(), torch.from_numpy(e).cuda()))
    o = dict(softcap=opts.get("softcap") or 0.0, logit_scale=opts.get("logit_scale", 1.0))
    want = ao.token_logprobs_grads(X, W, B, T, g.astype(np.float64), e.astype(np.float64), **o)
    # entries of the logit gradient and how far each may be off: its type's rounding (or the 2^-24 chain of
    # the fp32 path), and p, log p and H moving with the logits' error
    logp, ent64, z, slope = ao.token_logprobs(X, W, B, T, **o)
    valid = T >= 0
    lse = z.max(axis=1) + np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1))
    l = z - lse[:, None]
    p = np.exp(l) * valid[:, None]
    a = np.abs(g)[:, None] * p + np.abs(e)[:, None] * p * (np.abs(l) + ent64[:, None])
    a[np.arange(n)[valid], T[valid]] += np.abs(g)[valid]
    ez = _bounds(X, W, B, dtype, dict(o))[:, None]
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[dtype]
    tiny = 2.0 ** -24 if dtype == "f16" else 0.0
    d_err = np.abs(slope) * (a * (half + (4 + 2 * np.abs(l)) * (ez + 16 * U32 * (1 + np.abs(z) + np.abs(l))))
                             + tiny * a.max())
    if o["softcap"]:     # softcap' = 4 r (1 - r), r off by 2^-23
        d_err += 8 * U32 * a * o["logit_scale"]
    d_abs = np.abs(slope) * a
    for name, gotten, ref, err, size in (
            ("hidden", got[0], want[0], d_err @ np.abs(W), d_abs @ np.abs(W)),
            ("weight", got[1], want[1], d_err.T @ np.abs(X), d_abs.T @ np.abs(X)),
            ("bias", got[2] if b is not None else None, want[2], d_err.sum(0), d_abs.sum(0))):
        if gotten is None:
            continue
        out = 1.01 * half * np.abs(ref) + (2.0 ** -25 if dtype == "f16" else 0.0)
        terms = 64 + (v if name == "hidden" else n) / (1 if dtype == "f32" else 16)   # fp32 accumulation
        assert np.all(np.abs(_np(gotten) - ref) <= err + out + terms * U32 * size), name


@pytest.mark.parametrize("which", ["logps", "entropy"])
def test_one_upstream_gradient_alone(flce_lib, which):
    import torch
    x, w, b, t = _tensors(300, 64, 1000, "f32", seed=5)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w, b)]
    lp, ent = flce_lib.token_logprobs(*leaves[:2], t.cuda(), leaves[2], return_entropy=True)
    z = torch.zeros(300, device="cuda")
    g = torch.randn(300, generator=torch.Generator().manual_seed(1)).cuda()
    one = torch.autograd.grad(lp if which == "logps" else ent, leaves, g, retain_graph=True)
    both = torch.autograd.grad((lp, ent), leaves, (g, z) if which == "logps" else (z, g))
    for a, c in zip(one, both):
        assert torch.equal(a, c)


def test_logprobs_are_the_negative_loss(flce_lib):
    import torch
    x, w, b, t = (a.cuda() for a in _tensors(500, 128, 3000, "bf16", seed=6))
    lp = flce_lib.token_logprobs(x, w, t, b, softcap=9.0)
    loss, _, _ = flce_lib.forward(x, w, t, b, softcap=9.0, reduction="none")
    assert torch.max(torch.abs(lp + loss)) <= 64 * U32 * 10      # two roundings apart, of values up to ~ 10


def test_near_certain_rows_keep_their_small_entropy(flce_lib):
    """Logits of 60 against 0: H = 4.6e-23 x ..., far below the rounding of lse - sum p z (60 x 2^-24)."""
    import torch
    h, v = 64, 300
    for top in (12.0, 30.0, 60.0):
        x = torch.zeros(2, h)
        x[:, 0] = 1.0
        w = torch.zeros(v, h)
        w[7, 0] = top
        lp, ent = flce_lib.token_logprobs(x.cuda(), w.cuda(), torch.tensor([7, 3]).cuda(), return_entropy=True)
        rest = (v - 1) * np.exp(-top)
        lse = np.log1p(rest)
        want_h = lse + top * rest / (1 + rest) if top < 30 else rest * (1 + top)
        assert abs(lp[1].item() - (-top - lse)) <= 8 * U32 * top
        if top < 16:     # 1 + rest - 1 keeps 2^-24 absolute; smaller rests vanish in l = 1 + rest
            # l >= 1 after the certain logit: every later addition rounds it by at most half a step of
            # [1, 2), 2^-24.  Additions that reach it: 16 of its lane's 32 logits, 1 of the lane's two
            # sums, 1 into the running sum, 2 between lanes, 1 between waves, 2 splits = 23; then the
            # logarithm, a division and two products of values below 0.03: less than one more.
            assert abs(ent[0].item() - want_h) <= 24 * U32 * (1 + want_h)
        else:
            assert 0 <= ent[0].item() <= want_h * (1 + 1e-4) and ent[0].item() >= top * rest * (1 - 1e-4)


def test_masked_vocabulary_and_masked_rows(flce_lib):
    """A bias of -inf (or the type's lowest value) takes entries out; ignored and out-of-range rows
    may hold NaN and infinities; a target that the bias masks has log p = -inf."""
    import torch
    n, h, v = 300, 64, 700
    x, w, b, t = _tensors(n, h, v, "f32", seed=8)
    out = np.random.default_rng(1).random(v) < 0.5
    out[:300] = True                                     # a whole vocabulary tile's wave block, and more
    keep = np.flatnonzero(~out)
    t = torch.from_numpy(np.where(t.numpy() < 0, -100, keep[t.numpy() % len(keep)]))
    t[5] = v + 3                                         # out of range: as ignored
    t[6] = int(np.flatnonzero(out)[0])                   # masked target
    dead = (t < 0) | (t >= v)
    dead_x = x.clone()
    dead_x[dead] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0]).repeat(h // 4)
    g, e = torch.randn(n, generator=torch.Generator().manual_seed(2)), torch.ones(n)
    e[6] = g[6] = 0.0
    results = []
    for low, xx in ((-float("inf"), dead_x), (-float("inf"), x), (torch.finfo(torch.float32).min, x)):
        bias = torch.where(torch.from_numpy(out), torch.tensor(low), b)
        leaves = [a.cuda().requires_grad_(True) for a in (xx, w, bias)]
        lp, ent = flce_lib.token_logprobs(*leaves[:2], t.cuda(), leaves[2], return_entropy=True)
        grads = torch.autograd.grad((lp, ent), leaves, (g.cuda(), e.cuda()))
        assert lp[6].item() < -1e37       # (a logit of the type's lowest value counts as -inf)
        results.append([lp[torch.arange(n) != 6], ent, *grads])
    for other in results[1:]:
        for a, c in zip(results[0], other):
            assert torch.equal(a, c)
    lp, ent, gx, gw, gb = results[0]
    T = np.where((t.numpy() >= v) | (np.arange(n) == 6), -100, t.numpy())
    want_lp, want_h, _, _ = ao.token_logprobs(_np(x), _np(w)[keep], _np(b)[keep],
                                              np.where(T >= 0, np.searchsorted(keep, T), -100))
    rows = np.arange(n) != 6
    assert np.all(np.abs(_np(lp) - want_lp[rows]) <= 300 * U32) and np.all(np.abs(_np(ent) - want_h)[rows] <= 3000 * U32)
    assert torch.all(gx[torch.nonzero(dead)[:, 0].cuda()] == 0) and torch.all(torch.isfinite(gw))
    assert torch.all(gw[torch.from_numpy(np.flatnonzero(out)).cuda()] == 0)
    assert torch.all(gb[torch.from_numpy(np.flatnonzero(out)).cuda()] == 0)


@pytest.mark.parametrize("n", [9, 40, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_capped_infinite_logits_are_the_cap(flce_lib, n, dtype):
    """cap tanh(-inf) = -cap: with the softcap a bias of -inf leaves an entry in, at the lowest
    logit, also where whole tiles hold nothing else."""
    import torch
    x, w, b, t = _tensors(n, 64, 5000, dtype, seed=n)
    low = np.random.default_rng(3).random(5000) < 0.3
    low[:2100] = True
    out = torch.from_numpy(low)
    bias = torch.where(out, torch.tensor(-float("inf"), dtype=b.dtype), b)
    lp, ent = flce_lib.token_logprobs(x.cuda(), w.cuda(), t.cuda(), bias.cuda(), softcap=2.0, return_entropy=True)
    want_lp, want_h, _, _ = ao.token_logprobs(_np(x), _np(w), _np(bias), t.numpy(), softcap=2.0)
    # as in _check_values; the capped entries are exact, |z| <= 2 and z.max - z.min <= 4
    ez = _bounds(_np(x), _np(w), _np(torch.where(out, torch.zeros_like(b), b)), dtype, dict(softcap=2.0))
    own = 8 * U32 * (2 + np.log(5000) + 1)
    valid = t.numpy() >= 0
    assert np.all(np.abs(_np(lp) - want_lp)[valid] <= (2 * ez + own)[valid])
    assert np.all(np.abs(_np(ent) - want_h)[valid] <= ((1 + 2 * (4 + np.log(5000))) * ez + 2 * own)[valid])


@pytest.mark.parametrize("cap", [None, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ignored_rows_hold_anything(flce_lib, cap, dtype):
    import torch
    x, w, b, t = _tensors(290, 64, 700, dtype, seed=18, ignored=0.3)
    bad = x.clone()
    bad[t < 0] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0]).repeat(16).to(x.dtype)
    got = []
    for xx in (x, bad):
        leaves = [a.cuda().requires_grad_(True) for a in (xx, w, b)]
        lp, ent = flce_lib.token_logprobs(*leaves[:2], t.cuda(), leaves[2], softcap=cap, return_entropy=True)
        got.append([lp, ent, *torch.autograd.grad((lp, ent), leaves, (torch.ones_like(lp), torch.ones_like(lp)))])
    assert all(torch.equal(a, c) for a, c in zip(*got)) and torch.isfinite(got[0][3]).all()


def test_nan_in_a_row_that_counts_shows(flce_lib):
    import torch
    for cap in (None, 5.0):
        x, w, b, t = _tensors(40, 64, 300, "bf16", seed=9, ignored=0.0)
        x[7, 3] = float("nan")
        leaves = [x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)]
        lp, ent = flce_lib.token_logprobs(*leaves, t.cuda(), softcap=cap, return_entropy=True)
        assert torch.isnan(lp[7]) and torch.isnan(ent[7]) and torch.isfinite(lp).sum() == 39
        gx, gw = torch.autograd.grad(lp.sum(), leaves)
        assert torch.all(torch.isnan(gx[7])) and torch.isfinite(gx).all(dim=1).sum() == 39
        assert torch.isnan(gw).any()


def test_every_logit_masked_gives_nan(flce_lib):
    import torch
    x, w, _, t = _tensors(3, 64, 300, "bf16", seed=9, ignored=0.0)
    b = torch.full((300,), -float("inf"), dtype=torch.bfloat16)
    lp, ent = flce_lib.token_logprobs(x.cuda(), w.cuda(), t.cuda(), b.cuda(), return_entropy=True)
    assert torch.isnan(lp).all() and torch.isnan(ent).all()


def test_empty_batch_and_status(flce_lib):
    import torch
    w = torch.randn(100, 64, device="cuda", requires_grad=True)
    x = torch.zeros(0, 64, device="cuda", requires_grad=True)
    lp = flce_lib.token_logprobs(x, w, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert lp.shape == (0,)
    gx, gw = torch.autograd.grad(lp.sum(), (x, w))
    assert gx.shape == (0, 64) and not torch.any(gw)
    p = flce_lib.make_params(4, 64, 100, dtype="f32", reduction="none")
    ws = torch.empty(flce_lib.flce_logprobs_workspace_size(p, 0), dtype=torch.uint8, device="cuda")
    out = torch.empty(3, 4, device="cuda")
    x = torch.randn(4, 64, device="cuda")
    for t, code in (([0, 99, -100, 3], 0), ([0, 100, -100, 3], flce_lib.FLCE_ERR_TARGET_OUT_OF_RANGE), ([1, 2, 3, 4], 0)):
        tt = torch.tensor(t, device="cuda")
        rc = flce_lib.flce_logprobs_forward(p, x.data_ptr(), w.data_ptr(), None, tt.data_ptr(), out[0].data_ptr(), None,
                                            out[2].data_ptr(), ws.data_ptr(), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and flce_lib.get_status(ws) == code


def test_targets_need_no_alignment(flce_lib):
    import torch
    x, w, b, t = (a.cuda() for a in _tensors(100, 64, 300, "bf16", seed=41))
    longer = torch.cat([t[:1], t])
    for dt in (torch.int64, torch.int32):
        got = flce_lib.token_logprobs(x, w, longer.to(dt)[1:], b)
        assert torch.equal(got, flce_lib.token_logprobs(x, w, t, b))


def test_gradients_against_differences(flce_lib):
    """(f(x + d) - f(x - d)) / 2 |d| along random directions of hidden, weight and bias, fp32: the values'
    rounding 32 x 2^-24 x 300 / 2^-6 = 0.04 of a sum over 60 rows, the third-order term 2^-12 / 6 x 60."""
    import torch
    n, h, v = 60, 64, 300
    x, w, b, t = _tensors(n, h, v, "f32", seed=11)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w, b)]
    g = torch.randn(n, generator=torch.Generator().manual_seed(3)).cuda()
    opts = dict(logit_scale=0.8, softcap=6.0, return_entropy=True)

    def f(a):
        lp, ent = flce_lib.token_logprobs(a[0], a[1], t.cuda(), a[2], **opts)
        return (g * lp).double().sum() + 0.5 * ent.double().sum()

    grads = torch.autograd.grad(f(leaves), leaves)
    eps = 2.0 ** -6
    for k in range(3):
        d = torch.randn(leaves[k].shape, generator=torch.Generator().manual_seed(k)).cuda()
        d /= d.norm()
        move = lambda s: [a.detach() + (s * eps * d if i == k else 0) for i, a in enumerate(leaves)]  # noqa: E731
        diff = (f(move(1)) - f(move(-1))).item() / (2 * eps)
        assert abs(diff - (grads[k].double() * d.double()).sum().item()) <= 0.06


def test_repeatable_on_two_streams_and_captured(flce_lib):
    import torch
    sets = []
    for seed in (1, 2):
        x, w, b, t = _tensors(700, 128, 5000, "bf16", seed=seed)
        sets.append(([a.cuda().requires_grad_(True) for a in (x, w, b)], t.cuda()))

    def step(s):
        (x, w, b), t = s
        lp, ent = flce_lib.token_logprobs(x, w, t, b, return_entropy=True)
        return [lp.detach(), ent.detach(), *torch.autograd.grad((lp, ent), (x, w, b), (torch.ones_like(lp), ent.detach()))]

    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = step(sets[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(a, c) for a, c in zip(got[k], want[k]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(sets[0])
    for rep in range(6):
        with torch.no_grad():
            sets[0][0][0].copy_(sets[rep % 2][0][0] * (1 + rep))
        ref = step(sets[0])
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs, ref)), rep


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ordinary_head_on_sampled_rows(flce_lib, dtype):
    """N = 2000, H = 2048, V = 32000 with planted targets: values of every 37th row in fp64."""
    import torch
    inp = si.make_inputs(2000, 2048, 32000, dtype=dtype, weight_std=0.02, bias_std=0.1, ignore_frac=0.05,
                         reduction="none", seed=12, plant_frac=0.5, plant_margin=8.0)
    W, X, B = (si.widen(inp[k], dtype) for k in ("weight", "hidden", "bias"))
    from gpu_helpers import to_device
    d = to_device(inp, dtype)
    lp, ent = flce_lib.token_logprobs(d["hidden"], d["weight"], d["targets"], d["bias"], return_entropy=True)
    rows = np.arange(0, 2000, 37)
    _check_values(_np(lp)[rows], _np(ent)[rows], X[rows], W, B, inp["targets"][rows], dtype, {})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_last_round_of_tiles_runs_small(flce_lib, dtype):
    """N = 300 or 512, V = 36000: 282 large tiles on 256 CUs, of which whole rounds run large and the rest of
    the vocabulary small, in splits of its own (seen in the workspace: 16 bytes per split and padded row; fp32
    would run all of N = 300 small)."""
    import torch
    n, h, v = 512 if dtype == "f32" else 300, 512, 36000
    x, w, b, t = _tensors(n, h, v, dtype, seed=21)
    t[:4] = torch.tensor([v - 1, 0, 33000, 32767])          # on both sides of the seam
    p = flce_lib.make_params(n, h, v, dtype=dtype, reduction="none")
    splits = (flce_lib.flce_logprobs_workspace_size(p, 0) - 256) / 16 / 512
    assert splits > 128, splits
    lp, ent = flce_lib.token_logprobs(x.cuda(), w.cuda(), t.cuda(), b.cuda(), return_entropy=True)
    rows = np.r_[0:4, 4:n:17]
    _check_values(_np(lp)[rows], _np(ent)[rows], _np(x)[rows], _np(w), _np(b), t.numpy()[rows], dtype, {})


@pytest.mark.parametrize("n,h,v", [(300, 64, 1000), (700, 264, 9000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_only_the_wanted_gradients(flce_lib, n, h, v, dtype):
    """A frozen head, frozen states, a frozen bias: the other gradients' bits stay."""
    import torch
    x, w, b, t = _tensors(n, h, v, dtype, seed=31)
    ones = torch.ones(n, device="cuda")

    def grads(wanted):
        leaves = [a.cuda().requires_grad_(k in wanted) for k, a in zip("xwb", (x, w, b))]
        lp, ent = flce_lib.token_logprobs(leaves[0], leaves[1], t.cuda(), leaves[2], return_entropy=True)
        got = torch.autograd.grad((lp, ent), [a for a in leaves if a.requires_grad], (ones, ones))
        return dict(zip((k for k in "xwb" if k in wanted), got))

    full = grads("xwb")
    for wanted in ("x", "w", "b", "xb", "xw"):
        got = grads(wanted)
        assert list(got) == list(wanted)
        for k in wanted:
            assert torch.equal(got[k], full[k]), (wanted, k)


@pytest.mark.parametrize("n,h,v", [(70, 64, 500), (700, 264, 9000)])
@pytest.mark.parametrize("gw_dtype", ["f32", "bf16", "f16"])
def test_accumulated_gradients(flce_lib, n, h, v, gw_dtype):
    """FLCE_ACCUMULATE_GRAD_WEIGHT / _BIAS and a weight gradient of another type, through the C entry points:
    fp32 sums of the contraction and the buffer's contents, rounded once."""
    import torch
    x, w, b, t = (a.cuda() for a in _tensors(n, h, v, "bf16", seed=33))
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[gw_dtype]
    P = lambda a: a.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    lp, ent, lse = (torch.empty(n, device="cuda") for _ in range(3))
    ones = torch.ones(n, device="cuda")

    def run(acc, gw_type, gw, gb):
        p = flce_lib.make_params(n, h, v, dtype="bf16", grad_weight_dtype=gw_type, reduction="none",
                                 accumulate_grad_weight=acc, accumulate_grad_bias=acc)
        ws = torch.empty(flce_lib.flce_logprobs_workspace_size(p, 1), dtype=torch.uint8, device="cuda")
        assert flce_lib.flce_logprobs_forward(p, P(x), P(w), P(b), P(t), P(lp), P(ent), P(lse), P(ws), ws.numel(), st) == 0
        gx = torch.empty(n, h, dtype=torch.bfloat16, device="cuda")
        assert flce_lib.flce_logprobs_backward(p, P(x), P(w), P(b), P(t), P(lse), P(ent), P(ones), P(ones), P(gx), P(gw),
                                               P(gb), P(ws), ws.numel(), st) == 0
        return gw, gb

    exact, gb0 = run(False, "f32", torch.empty(v, h, device="cuda"), torch.empty_like(b))
    rounded, _ = run(False, gw_dtype, torch.empty(v, h, dtype=dt, device="cuda"), torch.empty_like(b))
    assert torch.equal(rounded, exact.to(dt))
    prior = torch.randn(v, h, device="cuda").to(dt)
    prior_b = torch.randn(v, device="cuda").bfloat16()
    gw, gb = run(True, gw_dtype, prior.clone(), prior_b.clone())
    assert torch.equal(gw, (exact + prior.float()).to(dt))
    assert torch.all((gb.float() - gb0.float() - prior_b.float()).abs() <= 2.0 ** -7 * (gb0.float().abs() + prior_b.float().abs()))


@pytest.mark.parametrize("n,h,v", [(1, 264, 900), (2, 64, 5001), (17, 136, 1100), (59, 520, 3350), (64, 72, 255)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_of_few_tokens_are_rounded_once(flce_lib, n, h, v, dtype):
    """Up to 64 tokens the logit gradient is held as a rounded value and the rest: 2^-17 (2^-23) of each entry.
    What is left: the outputs' own rounding, half a step; the softmax's fp32 (p, log p and H off by
    (4 + 2 |log p|) (z's bound + 16 x 2^-24 (1 + |z| + |log p|))) and the fp32 sums, as in
    test_values_and_gradients."""
    import torch
    x, w, b, t = _tensors(n, h, v, dtype, seed=77, ignored=0.0)
    leaves = [a.cuda().requires_grad_(True) for a in (x, w)]
    lp, ent = flce_lib.token_logprobs(*leaves, t.cuda(), return_entropy=True, vocab_chunk=1024)
    rng = np.random.default_rng(n)
    g, e = rng.normal(size=n).astype(np.float32), 0.1 * rng.normal(size=n).astype(np.float32)
    e = e.astype(np.float32)
    got = torch.autograd.grad((lp, ent), leaves, (torch.from_numpy(g).cuda(), torch.from_numpy(e).cuda()))
    X, W, T = _np(x), _np(w), t.numpy()
    want = ao.token_logprobs_grads(X, W, None, T, g.astype(np.float64), e.astype(np.float64))
    _, ent64, z, _ = ao.token_logprobs(X, W, None, T)
    l = z - (z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)))[:, None]
    p = np.exp(l)
    a = np.abs(g)[:, None] * p + np.abs(e)[:, None] * p * (np.abs(l) + ent64[:, None])
    a[np.arange(n), T] += np.abs(g)
    ez = _bounds(X, W, None, dtype, {})[:, None]
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    tiny = 2.0 ** -24 * a.max() if dtype == "f16" else 0.0      # the rest of an entry below fp16's normal range
    d_err = a * (half ** 2 / 2 + (4 + 2 * np.abs(l)) * (ez + 16 * U32 * (1 + np.abs(z) + np.abs(l)))) + tiny
    for name, gotten, ref, err, size in (("hidden", got[0], want[0], d_err @ np.abs(W), a @ np.abs(W)),
                                         ("weight", got[1], want[1], d_err.T @ np.abs(X), a.T @ np.abs(X))):
        out = 1.01 * half * np.abs(ref) + (2.0 ** -25 if dtype == "f16" else 0.0)
        assert np.all(np.abs(_np(gotten) - ref) <= out + err + (64 + v / 16) * U32 * size), name
