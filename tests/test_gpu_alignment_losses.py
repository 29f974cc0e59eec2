"""preference_loss and policy_loss on the GPU against the fp64 oracle.

Tolerances, before any run: per token the kernels do a handful of fp32 operations
(a difference, one or two exponentials of at most 1 ulp, two products), each within
2^-24 of its terms, the exponent's argument |logp - old| <= ~2 adding its own
rounding; so 16 x 2^-24 of the sum of the absolute terms bounds a token's loss and
gradient, before the output's own rounding (half a step of its type, at most
eps / 2 of the value, or half of a subnormal's step).  Sums are fp64."""
import numpy as np
import pytest

from oracle import alignment_oracle as ao

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _half_step(dtype, want):
    import torch
    fi = torch.finfo(dtype)
    return np.abs(want) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2


def _np(t):
    import torch
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def _make(layout, s, length, dtype, seed, poison=True):
    """Token tensors (as the layout lays them out), offsets and mask; masked tokens hold NaN,
    infinities and the type's lowest value."""
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = _dt(dtype)
    off = None
    shape = (s, length)
    if layout.startswith("packed"):
        lens = torch.randint(0, length + 1, (s,), generator=g)
        if s:
            lens[s // 2] = 0                       # an empty sequence
        off = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]) + (3 if "shift" in layout else 0)
        shape = (int(off[-1]) + 5,)                # tokens behind the last sequence
    mask = torch.rand(shape, generator=g) < 0.75
    if layout.startswith("padded") and s > 1:
        mask[s - 1] = False                        # a row that the mask leaves empty
    dead = ~mask
    if off is not None:
        at = torch.arange(shape[0])
        dead = dead | (at < off[0]) | (at >= off[-1])

    def place(x):
        if poison:
            bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dt).min])
            x = torch.where(dead, bad[torch.arange(x.numel()).reshape(shape) % 4].to(x.dtype), x)
        x = x.to(dt)
        if layout == "padded_sliced":              # rows of a longer buffer, from its second token on
            wide = torch.full((s, length + 3), 7.0, dtype=dt)
            wide[:, 1:length + 1] = x
            return wide.cuda()[:, 1:length + 1]
        return x.cuda()

    base = torch.log(torch.rand(shape, generator=g).clamp_min(1e-4))
    t = dict(logps=place(base), old=place(base + 0.3 * torch.randn(shape, generator=g)),
             ref=place(base + 0.3 * torch.randn(shape, generator=g)),
             entropy=place(2 * torch.rand(shape, generator=g)))
    if off is not None:
        t["offsets"] = off.to(torch.int32 if "i32" in layout else torch.int64).cuda()
    else:
        t["offsets"] = None
    t["mask"] = mask.cuda()
    t["noise"] = lambda *sh: torch.randn(*sh, generator=g)
    return t


SHAPES = [("padded", 2, 1), ("padded", 8, 300), ("padded", 6, 1027), ("padded", 2, 5000), ("padded", 64, 7),
          ("padded_sliced", 6, 515), ("padded", 4, 512), ("packed", 2, 1), ("packed", 10, 400),
          ("packed_i32_shift", 8, 3000), ("packed", 700, 5), ("packed_i32", 300, 1)]


@pytest.mark.parametrize("layout,s,length", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_preference_matches_the_oracle(flce_lib, layout, s, length, dtype):
    import torch
    t = _make(layout, s, length, dtype, seed=s * 1000 + length)
    lp = t["logps"].requires_grad_(True)
    off = None if t["offsets"] is None else t["offsets"].cpu().numpy().astype(np.int64)
    for kind, opts in (("sigmoid", dict(label_smoothing=0.1)), ("sigmoid", dict(margin=0.5)),
                       ("hinge", dict(length_normalize=True)), ("squared", dict(margin=-0.3))):
        for reduction in ("none", "mean", "sum"):
            opts = dict(opts, beta=0.2, loss_type=kind, reduction=reduction)
            ref = t["ref"] if kind != "hinge" else None
            loss, met = flce_lib.preference_loss(lp, ref, offsets=t["offsets"], mask=t["mask"], return_metrics=True,
                                                 **opts)
            g = t["noise"](s // 2) if reduction == "none" else torch.tensor(1.5)
            grad, = torch.autograd.grad(loss, lp, g.cuda())
            want, rewards, dgrad = ao.preference(_np(lp), _np(ref), off, t["mask"].cpu().numpy(), **opts)
            # rewards: sums of up to 5000 differences, each rounded once in fp32 (|logp - ref| < 16),
            # beta 0.2, then one fp32 rounding of the sum
            slack = 0.2 * length * 16 * U32 + 2 * U32 * np.abs(rewards).max(initial=0)
            got = np.concatenate([_np(met["chosen_rewards"]), _np(met["rejected_rewards"])])
            assert np.all(np.abs(got - rewards) <= slack), (kind, reduction)
            steep = 1.0 if kind != "squared" else 2 * (np.abs(rewards).max(initial=0) * 2 + 1) / 0.2 ** 2
            total = slack * 2 * steep * (s // 2 if reduction == "sum" else 1) + 2 * U32 * np.abs(want).max(initial=0)
            assert np.all(np.abs(_np(loss) - want) <= total), (kind, reduction)
            wg = dgrad(g.numpy())
            # the slope moves by at most (1, or 2 / beta^2 for the square) x the margin's error
            wobble = 0.2 * np.abs(_np(g)).max(initial=0) * (2 / 0.2 ** 2 if kind == "squared" else 1) * 2 * slack
            assert np.all(np.abs(_np(grad) - wg) <= wobble + 8 * U32 * np.abs(wg) + 1.01 * _half_step(lp.dtype, wg))


@pytest.mark.parametrize("layout,s,length", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_policy_matches_the_oracle(flce_lib, layout, s, length, dtype):
    import torch
    t = _make(layout, s, length, dtype, seed=s * 999 + length)
    lp, ent = t["logps"].requires_grad_(True), t["entropy"].requires_grad_(True)
    off = None if t["offsets"] is None else t["offsets"].cpu().numpy().astype(np.int64)
    mask = t["mask"].cpu().numpy()
    shape = tuple(lp.shape)
    for reduction in ("none", "sum", "mean", "sequence_mean"):
        for per_seq, full in ((True, True), (False, True), (True, False)):
            opts = dict(clip_low=0.2, clip_high=0.3, reduction=reduction)
            adv = t["noise"](s, 1) if per_seq else t["noise"](*shape)
            if full:
                opts.update(dual_clip=1.5, kl_coef=0.1, entropy_coef=0.05)
            loss, met = flce_lib.policy_loss(lp, t["old"], adv.cuda(), ref_logps=t["ref"] if full else None,
                                             entropy=ent if full else None, offsets=t["offsets"], mask=t["mask"],
                                             return_metrics=True, **opts)
            g = t["noise"](*shape) if reduction == "none" else torch.tensor(0.7)
            if reduction == "none":
                g = torch.where(torch.from_numpy(np.isfinite(_np(lp))), g, float("nan"))   # at masked places
            grads = torch.autograd.grad(loss, (lp, ent) if full else (lp,), g.cuda())
            want = ao.policy(_np(lp), _np(t["old"]), _np(adv), _np(t["ref"]) if full else None,
                             _np(ent) if full else None, off, mask, **opts)
            terms = want["terms"]
            tol = 16 * U32 * (terms if reduction == "none" else terms.sum())
            got = _np(loss)
            if not np.all(np.isfinite(want["loss"])):
                assert np.isnan(got) and want["num_tokens"] == 0
            else:
                assert np.all(np.abs(got - want["loss"]) <= tol + U32 * np.abs(want["loss"])), (reduction, per_seq)
            up = np.where(np.isnan(g.numpy()), 0, g.numpy())
            wg = want["grad"](up)
            assert np.all(np.abs(_np(grads[0]) - wg)
                          <= 16 * U32 * np.abs(up) * terms + 1.01 * _half_step(lp.dtype, wg)), (reduction, per_seq)
            if full:
                we = want["grad_entropy"](up)
                assert np.all(np.abs(_np(grads[1]) - we) <= 4 * U32 * np.abs(we) + 1.01 * _half_step(lp.dtype, we))
            assert met["num_tokens"].item() == want["num_tokens"]
            if want["num_tokens"]:
                assert abs(met["clip_fraction"].item() - want["clip_fraction"]) <= U32
                assert abs(met["kl"].item() - want["kl"]) <= 16 * U32 * (want["kl"] + 1)
            else:
                assert not np.any(wg) and np.isnan(met["clip_fraction"].item())


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens_at_all(flce_lib, packed):
    import torch
    off = torch.zeros(3, dtype=torch.int64, device="cuda") if packed else None
    lp = torch.zeros((0,) if packed else (2, 0), device="cuda", requires_grad=True)
    loss = flce_lib.preference_loss(lp, offsets=off)
    assert abs(loss.item() - np.log(2.0)) <= 2 * U32       # a margin of 0
    assert torch.autograd.grad(loss, lp)[0].shape == lp.shape
    adv = torch.ones(2, 1, device="cuda")
    for reduction, want in (("mean", np.nan), ("sequence_mean", np.nan), ("sum", 0.0)):
        loss = flce_lib.policy_loss(lp, lp.detach(), adv, offsets=off, reduction=reduction)
        assert np.array_equal(_np(loss), want, equal_nan=True)
        assert torch.autograd.grad(loss, lp)[0].shape == lp.shape
    none = torch.zeros((0,) if packed else (0, 3), device="cuda")
    off = torch.zeros(1, dtype=torch.int64, device="cuda") if packed else None
    assert np.isnan(flce_lib.preference_loss(none, offsets=off).item())
    assert flce_lib.preference_loss(none, offsets=off, reduction="none").shape == (0,)
    assert flce_lib.policy_loss(none, none, none if not packed else torch.zeros(0, 1, device="cuda"), offsets=off,
                                reduction="sum").item() == 0.0


def test_packed_buffer_without_a_sequence_gets_zero_gradients(flce_lib):
    import torch
    lp = torch.full((700,), float("nan"), device="cuda", requires_grad=True)
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    loss = flce_lib.policy_loss(lp, lp.detach(), torch.zeros(0, 1, device="cuda"), offsets=off, reduction="sum")
    assert loss.item() == 0.0 and torch.equal(torch.autograd.grad(loss, lp)[0], torch.zeros(700, device="cuda"))


def test_extreme_ratios(flce_lib):
    """Overflowed ratios, exact zeros and a certain reference (all in kept places)."""
    import torch
    inf = float("inf")
    lp = torch.tensor([[0.0, 0.0, 0.0, -inf, -200.0, 0.0]], device="cuda", requires_grad=True)
    old = torch.tensor([[-200.0, -200.0, -200.0, 0.0, 0.0, 0.0]], device="cuda")
    adv = torch.tensor([[1.0, 0.0, -1.0, 1.0, -1.0, 1.0]], device="cuda")
    loss = flce_lib.policy_loss(lp, old, adv, clip_low=0.25, clip_high=0.5, reduction="none")
    assert loss.tolist() == [[-1.5, 0.0, inf, 0.0, 0.75, -1.0]]
    loss = flce_lib.policy_loss(lp, old, adv, clip_low=0.25, clip_high=0.5, dual_clip=4.0, reduction="none")
    assert loss.tolist() == [[-1.5, 0.0, 4.0, 0.0, 0.75, -1.0]]
    grad, = torch.autograd.grad(loss, lp, torch.ones_like(loss))
    assert grad.tolist() == [[0.0, 0.0, 0.0, 0.0, 0.0, -1.0]]
    # ratios exactly on the border of a clip of nothing count as unclipped
    one = flce_lib.policy_loss(lp[:, 5:], old[:, 5:], adv[:, 5:], clip_low=0.0, clip_high=0.0)
    assert torch.autograd.grad(one, lp)[0][0, 5].item() == -1.0
    h = flce_lib.preference_loss(torch.tensor([[1e4], [-1e4]], device="cuda"), beta=1.0)
    assert h.item() == 0.0
    h = flce_lib.preference_loss(torch.tensor([[-1e4], [1e4]], device="cuda"), beta=1.0)
    assert h.item() == 2e4


def test_small_divergences_keep_their_digits(flce_lib):
    """k = e^d - d - 1 near 0, where the difference itself would lose them: 8 x 2^-24 of the value."""
    import torch
    d = torch.logspace(-6, 1.5, 1999, dtype=torch.float64)
    d = torch.cat([d, -d]).float()
    lp = torch.zeros(1, d.numel(), device="cuda")
    loss = flce_lib.policy_loss(lp, lp, lp, ref_logps=d[None].cuda(), kl_coef=1.0, reduction="none")
    x = d.double().numpy()
    want = np.where(np.abs(x) < 0.1, x * x * (1 / 2 + x * (1 / 6 + x * (1 / 24 + x * (1 / 120 + x * (1 / 720 + x / 5040))))),
                    np.expm1(x) - x)
    # the series is truncated at d^9 and expm1 - d loses at most a factor e^0.5 / 0.1487 at the seam
    assert np.all(np.abs(loss.cpu().numpy()[0] - want) <= 8 * U32 * want)


def test_long_sums_do_not_lose_the_margin(flce_lib):
    """Without a reference the reward is a sum of 200000 terms near -3: fp64 keeps its difference."""
    import torch
    n = 200_000
    lp = -3.0 + 0.01 * torch.randn(2, n, generator=torch.Generator().manual_seed(5))
    loss, met = flce_lib.preference_loss(lp.cuda(), beta=1.0, return_metrics=True)
    h = lp[0].double().sum() - lp[1].double().sum()
    want = np.logaddexp(0.0, -h.item())
    assert abs(loss.item() - want) <= 2 * U32 * abs(want) + 1e-9


def test_a_long_sequence_is_spread_and_bitwise_repeatable(flce_lib):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    t = 3_000_001
    lp = -torch.rand(t, generator=g, device="cuda")
    off = torch.tensor([0, 1, 2_900_000, 2_900_000, t], device="cuda")
    adv = torch.randn(4, 1, generator=g, device="cuda")
    runs = []
    for _ in range(3):
        x = lp.clone().requires_grad_(True)
        loss = flce_lib.policy_loss(x, lp + 0.1, adv, offsets=off, reduction="sequence_mean")
        both = flce_lib.preference_loss(x, offsets=off, beta=1e-6)
        runs.append((loss.detach(), *torch.autograd.grad(loss + both, x)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    want = ao.policy(_np(lp), _np(lp + 0.1), _np(adv), None, None, off.cpu().numpy(), reduction="sequence_mean")
    assert abs(runs[0][0].item() - want["loss"]) <= 16 * U32 * want["terms"].sum()


def test_two_streams_at_once_and_graph_replays(flce_lib):
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)

    def batch():
        lp = torch.log(torch.rand(64, 777, generator=g, device="cuda").clamp_min(1e-4))
        return dict(lp=lp.requires_grad_(True), old=(lp.detach() + 0.2 * torch.randn(64, 777, generator=g, device="cuda")),
                    adv=torch.randn(64, generator=g, device="cuda"), mask=torch.rand(64, 777, generator=g, device="cuda") < 0.8)

    def step(b):
        loss = flce_lib.policy_loss(b["lp"], b["old"], b["adv"], mask=b["mask"], reduction="sequence_mean")
        pref = flce_lib.preference_loss(b["lp"], b["old"], mask=b["mask"])
        return [loss.detach(), pref.detach(), torch.autograd.grad(loss + pref, b["lp"])[0]]

    a, b = batch(), batch()
    want = [step(a), step(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for k, x in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k] = step(x)
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(x, y) for x, y in zip(got[k], want[k]))
    graphs, outs = [], []
    for x in (a, b):          # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(x))
        graphs.append(graph)
    for rep in range(6):
        k = rep % 2
        if rep == 4:          # new contents between replays
            with torch.no_grad():
                a["lp"].mul_(1.1)
            want[0] = step(a)
        for o in outs[k]:
            o.fill_(-7)
        torch.cuda.synchronize()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs[k], want[k])), rep


def test_gradients_against_differences(flce_lib):
    """Through the torch op itself: (f(x + e) - f(x - e)) / 2e of the fp32 loss, e = 2^-6.
    Truncation e^2/6 x third derivative (< 3 per token here) <= 2e-4; rounding 2^-24 x |loss| (< 8)
    / 2^-6 <= 4e-5."""
    import torch
    gen = torch.Generator().manual_seed(9)
    lp = 0.3 * torch.randn(4, 3, generator=gen)
    old, ref = lp + 0.01, lp + 0.3 * torch.randn(4, 3, generator=gen)
    adv = torch.randn(4, 3, generator=gen)
    eps = 2.0 ** -6

    def f(x):
        x = x.cuda()
        return (flce_lib.policy_loss(x, old.cuda(), adv.cuda(), ref_logps=ref.cuda(), kl_coef=0.5, reduction="sum",
                                     clip_low=0.9, clip_high=9.0)
                + flce_lib.preference_loss(x, ref.cuda(), beta=0.7, reduction="sum"))

    x = lp.cuda().requires_grad_(True)
    grad, = torch.autograd.grad(f(x), x)
    for i in range(4):
        for j in range(3):
            d = torch.zeros(4, 3)
            d[i, j] = eps
            diff = (f(lp + d).item() - f(lp - d).item()) / (2 * eps)
            assert abs(diff - grad[i, j].item()) <= 4e-4


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean", "none"])
def test_gradients_of_one_input_alone(flce_lib, reduction):
    """Only the entropies, or only the log-probabilities, take part in autograd: the same bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    lp, ent = -torch.rand(5, 333, generator=g, device="cuda"), torch.rand(5, 333, generator=g, device="cuda")
    adv, mask = torch.randn(5, 333, generator=g, device="cuda"), torch.rand(5, 333, generator=g, device="cuda") < 0.6

    def grads(a, b):
        x, y = lp.clone().requires_grad_(a), ent.clone().requires_grad_(b)
        loss = flce_lib.policy_loss(x, lp + 0.1, adv, entropy=y, entropy_coef=0.3, mask=mask, reduction=reduction)
        return torch.autograd.grad(loss.sum(), [t for t in (x, y) if t.requires_grad])

    both = grads(True, True)
    assert torch.equal(grads(True, False)[0], both[0]) and torch.equal(grads(False, True)[0], both[1])
    with torch.no_grad():
        loss = flce_lib.policy_loss(lp.requires_grad_(True), lp + 0.1, adv, mask=mask)
    assert not loss.requires_grad
    with pytest.raises(RuntimeError):      # there is no second derivative
        x = lp.detach().clone().requires_grad_(True)
        d, = torch.autograd.grad(flce_lib.policy_loss(x, lp.detach(), adv), x, create_graph=True)
        torch.autograd.grad(d.sum(), x)


def test_as_many_packed_tokens_as_sequences(flce_lib):
    """(S,) advantages are per token or per sequence as the caller says: sequences of 0, 3, 1 and 0 tokens."""
    import torch
    lp = torch.tensor([-1.0, -2.0, -0.5, -3.0], device="cuda")
    old, adv = lp - 0.1, torch.tensor([1.0, -2.0, 3.0, -4.0], device="cuda")
    off = torch.tensor([0, 0, 3, 4, 4], device="cuda")
    for flag, want in ((True, [-2.0, -2.0, -2.0, 3.0]), (False, [1.0, -2.0, 3.0, -4.0])):
        loss = flce_lib.policy_loss(lp, old, adv, offsets=off, reduction="none", advantages_per_sequence=flag)
        assert torch.allclose(loss, -torch.tensor(want, device="cuda") * torch.exp(lp - old), rtol=1e-6)
    loss = flce_lib.policy_loss(lp, old, adv[:, None], offsets=off, reduction="none")
    assert torch.equal(loss, flce_lib.policy_loss(lp, old, adv, offsets=off, reduction="none",
                                                  advantages_per_sequence=True))
    one = flce_lib.policy_loss(lp[:1], old[:1], adv[:1], offsets=torch.tensor([0, 1], device="cuda"))
    assert torch.allclose(one, -torch.exp(lp[0] - old[0]), rtol=1e-6)


@pytest.mark.parametrize("s", [6, 200])
def test_offsets_against_the_rules_stay_inside_the_buffers(flce_lib, s):
    """Decreasing, negative and too large offsets: some answer, and zero gradients outside [first, last)."""
    import torch
    t = 3000
    g = torch.Generator().manual_seed(s)
    lp = (-torch.rand(t, generator=g)).cuda().requires_grad_(True)
    adv = torch.randn(s, 1, generator=g).cuda()
    for k in range(4):
        off = torch.randint(-2 * t, 3 * t, (s + 1,), generator=g)
        off[0], off[-1] = 100 * k, t - 50 * k
        loss = flce_lib.policy_loss(lp, lp.detach() - 0.1, adv, offsets=off.cuda(), reduction="sequence_mean")
        pref = flce_lib.preference_loss(lp, offsets=off.cuda())
        for grad in (torch.autograd.grad(loss, lp)[0], torch.autograd.grad(pref, lp)[0]):
            assert not torch.any(grad[:100 * k]) and not torch.any(grad[t - 50 * k:])
