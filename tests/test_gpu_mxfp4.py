"""MXFP4 quantisation and scores on the GPU.

Codes and scales are defined exactly and have to be equal.  A logit's sum is formed by matrix instructions that add
128 exact products to an fp32 sum: |error| <= 2 u (H / 128 + 8) sum_k |a_k b_k| (u = 2^-24; twice, for sums that are
cut off rather than rounded), then 5 roundings of at most u (|product| + |bias|) |scale|, the softcap's 3 u cap; the
softmax adds what test_gpu_token_logprobs.py derives."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao
from oracle import mx_oracle as mo

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _np(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (300, 1056), (3, 8192), (2, 1 << 18)])
def test_quantize_gives_the_defined_codes(flce_lib, dtype, rows, cols):
    import torch
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(getattr(torch, dtype))
    if rows >= 5:
        x[1] = 0.0
        x[2, 3] = float("nan")
        x[3, cols - 1] = -float("inf")
        x[4] = x[4].float().mul(1e-6).to(x.dtype)
    q, s = flce_lib.quantize_mxfp4(x.cuda())
    code, ws = mo.quantize(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), mo.pack(code))
    back = flce_lib.dequantize_mxfp4(q, s)
    assert np.array_equal(_np(back), mo.values(code, ws), equal_nan=True)


def test_every_16_bit_value(flce_lib):
    """All bf16 and fp16 values, in blocks whose scale is set by one large value of each power: every tie, both signs,
    subnormals, the least and greatest scales."""
    import torch
    bits = torch.arange(1 << 16, dtype=torch.int32)
    for dtype, tops in ((torch.bfloat16, [2.0 ** e for e in (-126, -125, -124, -60, -2, 0, 1, 2, 3, 60, 126, 127)]),
                        (torch.float16, [2.0 ** e for e in (-24, -14, -3, 0, 1, 2, 3, 15)])):
        x = bits.to(torch.int16).view(dtype)
        x = x[torch.isfinite(x)]
        for top in tops:
            near = x[x.double().abs() <= 2 * top]
            near = near[: near.numel() // 31 * 31].view(-1, 31)
            blocks = torch.cat([torch.full((near.shape[0], 1), top, dtype=dtype), near], 1)
            q, s = flce_lib.quantize_mxfp4(blocks.cuda())
            code, ws = mo.quantize(blocks.double().numpy())
            assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), mo.pack(code)), (dtype, top)


def test_fp32_extremes(flce_lib):
    import torch
    g = torch.Generator().manual_seed(3)
    x = torch.randn(64, 64, generator=g) * torch.exp2(torch.arange(64.0)[:, None] * 4 - 149 + 20)
    x[0] = torch.tensor([1e-45, -1e-45] * 32)
    x[1, 0] = torch.finfo(torch.float32).max
    x[2, 5] = torch.finfo(torch.float32).tiny
    q, s = flce_lib.quantize_mxfp4(x.cuda())
    code, ws = mo.quantize(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), mo.pack(code))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_dequantize_every_code_and_scale(flce_lib, dtype):
    """Every scale byte with every code, rounded once to the type (fp16: to infinity past its range)."""
    import torch
    dt = getattr(torch, dtype)
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    s = np.arange(256, dtype=np.uint8)[:, None]
    got = flce_lib.dequantize_mxfp4(torch.from_numpy(mo.pack(code)).cuda(), torch.from_numpy(s).cuda(), dtype=dt).cpu()
    want = torch.from_numpy(mo.values(code, s)).to(torch.float32).to(dt)      # fp32 holds them all
    assert got.dtype == dt and torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


def _problem(n, h, v, seed, ignored=0.1, bias=True, dtype="bfloat16"):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(n, h)) * np.exp(rng.normal(size=(n, 1)) * 0.3)).to(getattr(torch, dtype))
    w = torch.from_numpy(rng.normal(size=(v, h)) / np.sqrt(h)).float()
    b = torch.from_numpy(rng.normal(size=v) * 0.3).float() if bias else None
    t = rng.integers(0, v, size=n)
    t[rng.random(n) < ignored] = -100
    return x, w, b, torch.from_numpy(t)


def _check(lp, ent, a, w, b, t, rows=slice(None), scale=1.0, cap=0.0):
    """a, w: the values that the codes stand for."""
    a, T = a[rows], t[rows]
    product, terms = a @ w.T, (np.abs(a) @ np.abs(w).T).max(axis=1)
    want_lp, want_h, z, _ = ao.token_logprobs(None, None, b, T, logit_scale=scale, softcap=cap, product=product)
    valid = (T >= 0) & (T < len(w))
    ez = abs(scale) * (2 * U32 * (a.shape[1] / 128 + 8) * terms
                       + 5 * U32 * (np.abs(product).max(axis=1) + (0 if b is None else np.abs(b).max()))) + 3 * U32 * cap
    own = 24 * U32 * (np.abs(z).max(axis=1) + np.log(len(w)) + 1)
    spread = 1 + 2 * (z.max(axis=1) - z.min(axis=1) + np.log(len(w)))
    assert np.all(np.abs(lp[rows] - want_lp)[valid] <= (2 * ez + own)[valid])
    assert np.all(np.abs(ent[rows] - want_h)[valid] <= (spread * ez + 2 * own)[valid])
    assert not lp[rows][~valid].any() and not ent[rows][~valid].any()


# 1 to 16 tokens, up to 64, more; vocabularies of one, ragged, many tiles; rows of scales of every length modulo 8
SIZES = [(1, 32, 1), (1, 64, 7), (4, 4096, 5000), (16, 96, 300), (17, 160, 65), (63, 2048, 1000), (64, 224, 4097),
         (65, 128, 333), (200, 1056, 2500), (256, 256, 256), (300, 512, 9000), (513, 2048, 1111), (1000, 96, 20011),
         (2048, 64, 4096)]


@pytest.mark.parametrize("n,h,v", SIZES)
def test_scores(flce_lib, n, h, v):
    x, w, b, t = _problem(n, h, v, seed=n + h + v)
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), return_entropy=True)
    _check(_np(lp), _np(ent), mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy())),
           b.double().numpy(), t.numpy())


@pytest.mark.parametrize("n,h,v", [(3, 256, 900), (40, 96, 3000), (333, 1024, 5003)])
@pytest.mark.parametrize("scale,cap,bias,dtype", [(0.7, 0.0, False, "float16"), (1.25, 30.0, True, "float32"),
                                                  (1.0, 3.0, False, "bfloat16")])
def test_scale_softcap_bias(flce_lib, n, h, v, scale, cap, bias, dtype):
    x, w, b, t = _problem(n, h, v, seed=n, bias=bias, dtype=dtype)
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.int().cuda(), None if b is None else b.cuda(),
                                            logit_scale=scale, softcap=cap or None, return_entropy=True)
    _check(_np(lp), _np(ent), mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy())),
           None if b is None else b.double().numpy(), t.numpy(), scale=scale, cap=cap)


@pytest.mark.parametrize("n,h,v", [(16, 4096, 128256), (1000, 2048, 50001), (4096, 512, 128256)])
def test_large_heads(flce_lib, n, h, v):
    """Sampled rows; the head's values come from the framework, whose codes the other tests pin."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(v)
    w = torch.randn(v, h, generator=g, device="cuda") / h ** 0.5
    x = torch.randn(n, h, generator=g, device="cuda").to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::9] = -100
    q, s = flce_lib.quantize_mxfp4(w)
    lp, ent = flce_lib.token_logprobs_mxfp4(x, q, s, t, return_entropy=True)
    rows = np.unique(np.linspace(0, n - 1, 12).astype(int))
    _check(_np(lp), _np(ent), mo.values(*mo.quantize(_np(x))), _np(flce_lib.dequantize_mxfp4(q, s)), None, _np(t).astype(int),
           rows=rows)


@pytest.mark.parametrize("n", [5, 100, 700])
def test_scales_of_all_sizes(flce_lib, n):
    """Blocks of very different powers within a row: each product carries both of its own scales."""
    import torch
    rng = np.random.default_rng(n)
    x, w, b, t = _problem(n, 512, 1500, seed=n)
    up = np.repeat(rng.integers(-20, 20, size=(n, 16)), 32, axis=1)
    down = np.repeat(rng.integers(-20, 0, size=(1500, 16)), 32, axis=1)
    x = (x.double() * torch.from_numpy(np.exp2(np.minimum(up, 0)))).float()
    w = (w.double() * torch.from_numpy(np.exp2(down / 4.0))).float()
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), return_entropy=True)
    _check(_np(lp), _np(ent), mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy())),
           b.double().numpy(), t.numpy())


@pytest.mark.parametrize("n", [3, 50, 600])
@pytest.mark.parametrize("h", [128, 160])
def test_quantized_states_and_slices(flce_lib, n, h):
    """States that are quantized already give the same bits; slices of a vocabulary, of rows that are not 16-byte
    aligned in their scales, give the slice's own log-probabilities."""
    import torch
    x, w, b, t = _problem(n, h, 2000, seed=n)
    x, w, b, t = x.cuda(), w.cuda(), b.cuda(), t.cuda()
    q, s = flce_lib.quantize_mxfp4(w)
    want = flce_lib.token_logprobs_mxfp4(x, q, s, t, b)
    assert torch.equal(flce_lib.token_logprobs_mxfp4(*(lambda a: (a[0], q, s, t, b))(flce_lib.quantize_mxfp4(x)),
                                                     hidden_scale=flce_lib.quantize_mxfp4(x)[1]), want)
    for first in (1, 3, 1001):
        part = flce_lib.token_logprobs_mxfp4(x, q[first:], s[first:], t % 900, b[first:])
        alone = flce_lib.token_logprobs_mxfp4(x, q[first:].clone(), s[first:].clone(), t % 900, b[first:].clone())
        assert torch.equal(part, alone)


@pytest.mark.parametrize("h", [224, 256])
def test_quantized_states_in_large_tiles(flce_lib, h):
    """Codes and scales that are given, in rows that need padding (7 scales) and in whole ones."""
    import torch
    x, w, b, t = _problem(1030, h, 9001, seed=h)
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    xq, xs = flce_lib.quantize_mxfp4(x.cuda())
    got = flce_lib.token_logprobs_mxfp4(xq, q, s, t.cuda(), b.cuda(), hidden_scale=xs, return_entropy=True)
    want = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), return_entropy=True)
    assert all(torch.equal(p, r) for p, r in zip(got, want))
    _check(_np(got[0]), _np(got[1]), mo.values(*mo.quantize(x.double().numpy())),
           mo.values(*mo.quantize(w.double().numpy())), b.double().numpy(), t.numpy())


@pytest.mark.parametrize("n", [7, 1500])
def test_scale_of_either_sign_and_zero(flce_lib, n):
    """A negative logit_scale turns the order of the logits round; with 0 every entry has the same probability."""
    import torch
    x, w, b, t = _problem(n, 128, 3003, seed=n, ignored=0.0)
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    values = mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy()))
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), logit_scale=-0.8, return_entropy=True)
    _check(_np(lp), _np(ent), *values, b.double().numpy(), t.numpy(), scale=-0.8)
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), logit_scale=0.0, return_entropy=True)
    want = np.log(3003.0)
    assert np.all(np.abs(_np(lp) + want) <= 48 * U32 * (want + 1)) and np.all(np.abs(_np(ent) - want) <= 48 * U32 * (want + 1))


@pytest.mark.parametrize("n", [4, 90, 600])
def test_masked_rows_and_entries(flce_lib, n):
    """NaN states of ignored rows stay there; targets out of range count as ignored; a bias of -inf takes entries out;
    a NaN state makes its own row NaN."""
    import torch
    x, w, b, t = _problem(n, 256, 1100, seed=n, ignored=0.0)
    x[1], t[1] = float("nan"), -100
    t[2] = 1100
    x[3, 40] = float("inf")
    t[3] = 5
    b[200:900] = -float("inf")
    t[0] = 950
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), b.cuda(), return_entropy=True)
    lp, ent = _np(lp), _np(ent)
    assert lp[1] == ent[1] == lp[2] == ent[2] == 0 and np.isnan(lp[3]) and np.isnan(ent[3])
    keep = np.r_[0:200, 900:1100]
    place = np.full(1100, -100)
    place[keep] = np.arange(len(keep))
    T = place[np.clip(t.numpy(), 0, 1099)]
    T[[1, 2, 3]] = -100
    rows = np.flatnonzero(T >= 0)
    assert 0 in rows
    _check(lp, ent, mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy()))[keep],
           b.double().numpy()[keep], T, rows=rows)


@pytest.mark.parametrize("n,v", [(4, 3003), (90, 3003), (1030, 9001)])
@pytest.mark.parametrize("bias", [False, True])
def test_logits_past_the_range(flce_lib, n, v, bias):
    """A logit whose products leave fp32's range downwards has probability 0, as has one with a bias of -inf (whole
    tiles of them here): the other entries' log-probabilities and the entropy are those without it."""
    import torch
    x, w, b, t = _problem(n, 128, v, seed=n, ignored=0.0, bias=bias)
    x, w = x.abs() + 1, w.clone()
    w[17] = -2.0 ** 127
    out = np.zeros(v, dtype=bool)
    out[17] = True
    if bias:
        out[100:900] = True
        b[100:900] = -float("inf")
    keep = np.flatnonzero(~out)
    place = np.cumsum(~out) - 1
    t[torch.from_numpy(out)[t]] = 18
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, t.cuda(), None if b is None else b.cuda(), return_entropy=True)
    _check(_np(lp), _np(ent), mo.values(*mo.quantize(x.double().numpy())), mo.values(*mo.quantize(w.double().numpy()))[keep],
           None if b is None else b.double().numpy()[keep], place[t.numpy()])


def test_no_tokens_and_all_ignored(flce_lib):
    import torch
    x, w, b, t = _problem(20, 64, 300, seed=1)
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    assert flce_lib.token_logprobs_mxfp4(x[:0].cuda(), q, s, t[:0].cuda()).shape == (0,)
    lp, ent = flce_lib.token_logprobs_mxfp4(x.cuda(), q, s, torch.full((20,), -100, device="cuda"), return_entropy=True)
    assert not lp.any() and not ent.any()
    q0, s0 = flce_lib.quantize_mxfp4(x[:0].cuda())
    assert q0.shape == (0, 32) and s0.shape == (0, 2) and flce_lib.dequantize_mxfp4(q0, s0).shape == (0, 64)


@pytest.mark.parametrize("n", [8, 300])
def test_replays_and_streams(flce_lib, n):
    """A captured call replayed on new inputs, and calls on another stream, give the eager bits."""
    import torch
    x, w, b, t = _problem(n, 512, 3001, seed=2)
    x, b, t = x.cuda(), b.cuda(), t.cuda()
    q, s = flce_lib.quantize_mxfp4(w.cuda())

    def call():
        return flce_lib.token_logprobs_mxfp4(x, q, s, t, b, softcap=20.0, return_entropy=True)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [call() for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, r) for out in got for p, r in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).to(x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(out, call()))


def test_gradients_and_tangents_are_refused(flce_lib):
    import torch
    import torch.autograd.forward_ad as fwAD
    x, w, b, t = _problem(4, 64, 40, seed=5)
    x, b, t = x.cuda(), b.cuda(), t.cuda()
    q, s = flce_lib.quantize_mxfp4(w.cuda())
    with pytest.raises(ValueError):
        flce_lib.token_logprobs_mxfp4(x.requires_grad_(True), q, s, t, b)
    with torch.no_grad():
        flce_lib.token_logprobs_mxfp4(x, q, s, t, b)
    with fwAD.dual_level(), torch.no_grad(), pytest.raises(ValueError):
        flce_lib.token_logprobs_mxfp4(fwAD.make_dual(x.detach(), torch.ones_like(x)), q, s, t, b)
    assert not flce_lib.quantize_mxfp4(x)[0].requires_grad
