"""quantize_int8 and token_logprobs_int8 on the GPU against the fp64 oracle.

The quantized integers and scales are defined by fp32 operations and have to be equal.
The scores' products are exact integers; a logit is one conversion, two products and an
addition, so |error| <= 5 x 2^-24 (|s_i s_j q_i . q_j| + |b_j|) |scale|, and the softmax
adds what test_gpu_token_logprobs.py derives."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _np(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (300, 1040), (3, 8192), (2, 131072)])
def test_quantize_gives_the_defined_integers(flce_lib, dtype, rows, cols):
    import torch
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(getattr(torch, dtype))
    if rows >= 5:
        x[1] = 0.0
        x[2, 3] = float("nan")
        x[3, cols - 1] = -float("inf")
        x[4] = 1e-38
    q, s = flce_lib.quantize_int8(x.cuda())
    wq, ws = ao.quantize_int8(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    if rows < 5:
        assert np.all(np.abs(x.double().numpy() - q.double().cpu().numpy() * _np(s)[:, None])
                      <= _np(s)[:, None] * (0.5 + 1e-4))


def _problem(n, h, v, seed, ignored=0.1, bias=True):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(n, h))).to(torch.bfloat16)
    w = torch.from_numpy(rng.normal(size=(v, h)) * 0.1)
    b = torch.from_numpy(rng.normal(size=v) * 0.3).float() if bias else None
    t = rng.integers(0, v, size=n)
    t[rng.random(n) < ignored] = -100
    return x, w.float(), b, torch.from_numpy(t)


def _check(lp, ent, q, s, wq, ws, b, t, rows=slice(None), scale=1.0, cap=0.0):
    product = (q[rows].astype(np.float64) @ wq.astype(np.float64).T) * s[rows, None] * ws[None]
    T = t[rows]
    want_lp, want_h, z, _ = ao.token_logprobs(None, None, b, T, logit_scale=scale, softcap=cap, product=product)
    valid = (T >= 0) & (T < len(ws))
    ez = 5 * U32 * abs(scale) * (np.abs(product).max(axis=1) + (0 if b is None else np.abs(b).max())) + 3 * U32 * cap
    own = 24 * U32 * (np.abs(z).max(axis=1) + np.log(len(ws)) + 1)
    spread = 1 + 2 * (z.max(axis=1) - z.min(axis=1) + np.log(len(ws)))
    assert np.all(np.abs(lp[rows] - want_lp)[valid] <= (2 * ez + own)[valid])
    assert np.all(np.abs(ent[rows] - want_h)[valid] <= (spread * ez + 2 * own)[valid])
    assert not np.any(lp[rows][~valid]) and not np.any(ent[rows][~valid])


SHAPES = [(1, 16, 1), (1, 64, 1000), (2, 48, 257), (7, 4096, 300), (16, 112, 513), (17, 128, 255), (33, 64, 2000),
          (64, 144, 1025), (65, 64, 700), (255, 64, 513), (256, 128, 512), (300, 272, 2049), (1030, 48, 1100)]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("opts", [dict(), dict(logit_scale=0.7, softcap=5.0)])
def test_scores_match_the_oracle(flce_lib, n, h, v, opts):
    import torch
    x, w, b, t = _problem(n, h, v, seed=n + h + v, bias=n % 2 == 0)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), None if b is None else b.cuda(),
                                           return_entropy=True, **opts)
    q, s = ao.quantize_int8(x.float().numpy())
    _check(_np(lp), _np(ent), q, s.astype(np.float64), wq.cpu().numpy(), _np(ws), None if b is None else _np(b),
           t.numpy(), scale=opts.get("logit_scale", 1.0), cap=opts.get("softcap") or 0.0)
    # the quantized form of the call, int32 targets, without entropies: the same bits
    again = flce_lib.token_logprobs_int8(torch.from_numpy(q).cuda(), wq, ws, t.int().cuda(),
                                         None if b is None else b.cuda(), hidden_scale=torch.from_numpy(s).cuda(), **opts)
    assert torch.equal(again, lp)


def test_largest_products_do_not_overflow(flce_lib):
    """All 127s at the largest hidden size: sums of 2^17 x 127^2 = 2.1e9 < 2^31."""
    import torch
    h = 1 << 17
    q = torch.full((3, h), 127, dtype=torch.int8)
    q[1] = -127
    wq = torch.full((20, h), 127, dtype=torch.int8)
    wq[10:] = -127
    s, ws = torch.full((3,), 2.0 ** -20), torch.full((20,), 2.0 ** -8)
    t = torch.tensor([3, 3, 15])
    lp = flce_lib.token_logprobs_int8(q.cuda(), wq.cuda(), ws.cuda(), t.cuda(), hidden_scale=s.cuda())
    z = 127.0 * 127.0 * h * 2.0 ** -28
    assert abs(lp[0].item() + np.log(10)) < 1e-4 and abs(lp[2].item() + 2 * z + np.log(10)) < 1e-4
    assert abs(lp[1].item() + 2 * z + np.log(10)) < 1e-4


def test_rows_that_hold_nan_and_zeros(flce_lib):
    import torch
    x, w, b, t = _problem(40, 64, 300, seed=3, ignored=0.0)
    x[3, 5] = float("nan")
    x[4] = 0.0
    t[5] = -100
    x[5] = float("inf")
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), return_entropy=True)
    assert torch.isnan(lp[3]) and lp[5] == 0 and ent[5] == 0 and torch.isfinite(lp).sum() == 39
    assert abs(lp[4].item() + np.log(300)) < 1e-5 and abs(ent[4].item() - np.log(300)) < 1e-5


def test_masked_vocabulary(flce_lib):
    import torch
    x, w, b, t = _problem(20, 64, 600, seed=4, ignored=0.0)
    out = torch.arange(600) % 3 == 0
    out[:260] = True
    t[:] = 300 + 1
    bias = torch.where(out, -float("inf"), b)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), bias.cuda(), return_entropy=True)
    keep = torch.nonzero(~out)[:, 0].cuda()
    want = flce_lib.token_logprobs_int8(x.cuda(), wq[keep].contiguous(), ws[keep].contiguous(),
                                        torch.full((20,), int((keep == 301).nonzero().item())).cuda(),
                                        bias.cuda()[keep].contiguous(), return_entropy=True)
    assert torch.allclose(lp, want[0], atol=64 * U32 * 10) and torch.allclose(ent, want[1], atol=64 * U32 * 10)


def test_scores_are_near_those_of_the_unquantized_head(flce_lib):
    """Quantization moves a logit by at most sum |x| s_w / 2 + |w| s_x / 2 (+ their product)."""
    x, w, b, t = _problem(200, 256, 3000, seed=5, ignored=0.0, bias=False)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp = _np(flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda()))
    X, W = _np(x), _np(w)
    q, s = ao.quantize_int8(x.float().numpy())
    sw = _np(ws)
    off = (np.abs(X).sum(1)[:, None] * sw[None] / 2 + np.abs(W).sum(1)[None] * s[:, None] / 2
           + 256 * s[:, None] * sw[None] / 4).max(axis=1) * 1.01
    want, _, _, _ = ao.token_logprobs(X, W, None, t.numpy())
    assert np.all(np.abs(lp - want) <= 2 * off)
    assert np.median(np.abs(lp - want)) < 0.1      # and in fact far less: the errors are random


def test_large_ragged_batch_on_sampled_rows(flce_lib):
    x, w, b, t = _problem(2111, 1024, 33001, seed=6)
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), b.cuda(), return_entropy=True)
    q, s = ao.quantize_int8(x.float().numpy())
    _check(_np(lp), _np(ent), q, s.astype(np.float64), wq.cpu().numpy(), _np(ws), _np(b), t.numpy(),
           rows=np.arange(0, 2111, 41))


def test_empty_batch_streams_and_capture(flce_lib):
    import torch
    x, w, b, t = (a.cuda() for a in _problem(500, 128, 4000, seed=7))
    wq, ws = flce_lib.quantize_int8(w)
    assert flce_lib.token_logprobs_int8(x[:0], wq, ws, t[:0]).shape == (0,)
    sets = [(x, t), (x.flip(0).contiguous(), t)]
    step = lambda k: flce_lib.token_logprobs_int8(sets[k][0], wq, ws, sets[k][1], b, return_entropy=True)  # noqa: E731
    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(4):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = step(k)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for k in (0, 1) for a, c in zip(got[k], want[k]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(0)
    for rep in range(6):
        sets[0][0].mul_(1.01)
        ref = step(0)
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs, ref)), rep


def test_last_round_of_tiles_runs_small(flce_lib):
    """As in test_gpu_token_logprobs.py: 282 large tiles, the last 26 of them run as small ones."""
    n, h, v = 300, 1024, 36000
    x, w, b, t = _problem(n, h, v, seed=22)
    t[0], t[1], t[2] = v - 1, 33000, 32767
    p = flce_lib.make_params(n, h, v, reduction="none")
    assert (flce_lib.flce_logprobs_int8_workspace_size(p) - 256) / 16 / 512 > 128
    wq, ws = flce_lib.quantize_int8(w.cuda())
    lp, ent = flce_lib.token_logprobs_int8(x.cuda(), wq, ws, t.cuda(), b.cuda(), return_entropy=True)
    q, s = ao.quantize_int8(x.float().numpy())
    _check(_np(lp), _np(ent), q, s.astype(np.float64), wq.cpu().numpy(), _np(ws), _np(b), t.numpy(),
           rows=np.r_[0:3, 3:300:17])
