"""The alignment-training operators as measurable cases: per-token log-probabilities of a linear head with their
gradients, the same scores from an 8-bit head, the paired preference loss and the clipped policy loss.

``own`` false: the operators in elementary torch operations.  ``own`` true: the framework's entry points."""
import math

import torch

own = False

SHARE_MASKED = 0.05          # rows whose target is ignored
BETA = 0.1


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # scoring the sampled tokens of one decoding step of a small batch
        dict(name="logprobs score n16", op="logprobs", dtype="bf16", n=16, h=4096, v=32000, bias=False, scale=1.0,
             cap=0.0, back=False),
        # a debugging run in single precision, odd sizes, bias and entropy bonus
        dict(name="logprobs train f32", op="logprobs", dtype="f32", n=515, h=1024, v=8191, bias=True, scale=1.0,
             cap=0.0, back=True),
        # a short fine-tuning step in half precision with a capped, tempered head
        dict(name="logprobs train f16", op="logprobs", dtype="f16", n=2001, h=2048, v=32000, bias=False, scale=0.7,
             cap=30.0, back=True),
        # the training step of a large head
        dict(name="logprobs train bf16", op="logprobs", dtype="bf16", n=8192, h=4096, v=128256, bias=False,
             scale=1.0, cap=0.0, back=True),
        # a frozen scorer's 8-bit head: the tokens of one decoding step
        dict(name="int8 score n4", op="int8", dtype="bf16", n=4, h=4096, v=128256, bias=False, scale=1.0, cap=0.0),
        # one ragged packed answer batch
        dict(name="int8 score n1000", op="int8", dtype="f16", n=1000, h=2048, v=50001, bias=True, scale=1.0,
             cap=30.0),
        # the reference's scores of a whole training batch
        dict(name="int8 score n8192", op="int8", dtype="bf16", n=8192, h=4096, v=128256, bias=False, scale=1.0,
             cap=0.0),
        # four pairs of short answers, packed
        dict(name="preference 4 pairs", op="preference", dtype="f32", seqs=8, length=300, packed=True,
             loss="sigmoid", smoothing=0.1, reference=True, normalize=False),
        # a large padded batch of pairs with prompts masked out
        dict(name="preference 1024 pairs", op="preference", dtype="f32", seqs=2048, length=2048, packed=False,
             loss="sigmoid", smoothing=0.0, reference=True, normalize=False),
        # one group of sampled answers
        dict(name="policy 16 answers", op="policy", dtype="f32", seqs=16, length=256, packed=False, reference=False,
             entropy=False, per_sequence=True, dual=False, reduction="mean"),
        # a packed batch of groups in 16 bits with a reference, averaged per answer
        dict(name="policy packed bf16", op="policy", dtype="bf16", seqs=513, length=1500, packed=True,
             reference=True, entropy=False, per_sequence=True, dual=False, reduction="sequence_mean"),
        # the full loss over a large padded batch of long answers
        dict(name="policy 2048 answers", op="policy", dtype="f32", seqs=2048, length=8192, packed=False,
             reference=True, entropy=True, per_sequence=False, dual=True, reduction="mean"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "int8", "preference", "policy"])
    if op in ("logprobs", "int8"):
        case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32", "bf16"]), n=_log_int(rng, 1, 8192),
                    h=16 * _log_int(rng, 8, 256), v=_log_int(rng, 500, 128256), bias=rng.random() < 0.4,
                    scale=rng.choice([1.0, 0.7, 1.25]), cap=rng.choice([0.0, 0.0, 30.0]))
        if op == "logprobs":
            case["back"] = rng.random() < 0.7
            if case["dtype"] == "f32":
                case["n"] = min(case["n"], 1 + case["n"] % 1024)
        return case
    seqs = _log_int(rng, 1, 1024) * 2
    length = _log_int(rng, 1, 8192)
    most = 4 << 20 if op == "preference" else 16 << 20
    length = max(1, min(length, most // seqs))
    case = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), seqs=seqs, length=length,
                packed=rng.random() < 0.5, reference=rng.random() < 0.7)
    if op == "preference":
        case.update(loss=rng.choice(["sigmoid", "hinge", "squared"]), normalize=rng.random() < 0.3)
        case["smoothing"] = rng.choice([0.0, 0.1]) if case["loss"] == "sigmoid" else 0.0
    else:
        case.update(entropy=rng.random() < 0.4, per_sequence=rng.random() < 0.5, dual=rng.random() < 0.4,
                    reduction=rng.choice(["mean", "sequence_mean", "sum", "none"]))
    return case


TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------------------- inputs

def _quantize(x):
    """Symmetric 8-bit rows, defined in 32 bits: s = max|x| * fp32(1/127), q = rint(x * fp32(1/s))."""
    x = x.float()
    s = x.abs().amax(1) * torch.tensor(1.0 / 127.0, dtype=torch.float32, device=x.device)
    r = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    return torch.round(x * r[:, None]).clamp(-127, 127).to(torch.int8), s


def _packed_tokens(case):
    return max(case["length"], int(0.6 * case["seqs"] * case["length"]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] in ("logprobs", "int8"):
        n, h, v, dt = case["n"], case["h"], case["v"], TORCH[case["dtype"]]
        w = torch.empty(v, h, dtype=torch.float32, device="cuda").normal_(0, 1 / math.sqrt(h), generator=g)
        targets = torch.randint(0, v, (n,), generator=g, device="cuda")
        # each token's state leans towards its target's row by its own amount: some tokens are almost sure, some not
        lean = rand(n, 1) * 1.5 * math.log(v)
        x = randn(n, h) + lean * w[targets]
        if n > 1:
            targets = torch.where(rand(n) < SHARE_MASKED, torch.full_like(targets, -100), targets)
        s["hidden"] = x.to(dt)
        s["targets"] = targets
        s["bias"] = (0.3 * randn(v)).to(torch.float32 if case["op"] == "int8" else dt) if case["bias"] else None
        if case["op"] == "int8":
            s["weight"], s["weight_scale"] = _quantize(w)     # laid out once, when the scorer is loaded
        else:
            s["weight"] = w.to(dt)
            if case["back"]:
                unit = (256.0 if case["dtype"] == "f16" else 1.0) / n      # half precision trains with a loss scale
                s["grad_logps"] = unit * randn(n)
                s["grad_entropy"] = 0.1 * unit * randn(n)
                for k in ("hidden", "weight", "bias"):
                    if s[k] is not None:
                        s[k].requires_grad_(True)
        return s
    b, length, dt = case["seqs"], case["length"], TORCH[case["dtype"]]
    lens = (length * rand(b).mul(1.3).sub(0.05).clamp(0, 1)).round().long()    # ragged, some full, a few empty
    lens[0] = length
    if case["packed"]:
        # one buffer of a fixed size for all batches: the answers fill most of it, or the last ones are cut
        shape = (_packed_tokens(case),)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)]).clamp(max=shape[0])
        s["mask"] = None
    else:
        prompt = (0.3 * rand(b) * lens).long()
        at = torch.arange(length, device="cuda")
        s["offsets"] = None
        s["mask"] = (at < lens[:, None]) & (at >= prompt[:, None])
        shape = (b, length)
    logps = torch.log(rand(*shape).clamp_min(1e-6)) * 1.2
    s["logps"] = logps.to(dt).requires_grad_(True)
    s["ref_logps"] = (logps + 0.2 * randn(*shape)).to(dt) if case["reference"] else None
    if case["op"] == "policy":
        s["old_logps"] = (logps + 0.15 * randn(*shape)).to(dt)
        s["advantages"] = randn(b) if case["per_sequence"] else randn(*shape)
        s["entropies"] = (2 * rand(*shape)).to(dt).requires_grad_(True) if case["entropy"] else None
        s["grad"] = rand(*shape) if case["reduction"] == "none" else torch.full((), 1.0, device="cuda")
    return s


def work(case):
    if case["op"] in ("logprobs", "int8"):
        n, h, v = case["n"], case["h"], case["v"]
        e = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
        back = case["op"] == "logprobs" and case["back"]
        we = 1 if case["op"] == "int8" else e
        by = n * h * e + v * h * we + 16 * n
        if back:
            by += n * h * e + v * h * e + 8 * n
        return {"bytes": by, "flops": 2.0 * n * h * v * (3 if back else 1)}
    t = _packed_tokens(case) if case["packed"] else case["seqs"] * case["length"]
    e = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    by = t * (e * (2 + int(case["reference"])) + (0 if case["packed"] else 1))     # log-probabilities in, gradient out
    if case["op"] == "preference":
        return {"bytes": by, "flops": 4.0 * t}
    by += t * (e + (0 if case["per_sequence"] else 4) + (2 * e if case["entropy"] else 0))
    by += t * (8 if case["reduction"] == "none" else 0)
    return {"bytes": by, "flops": 20.0 * t}


# ----------------------------------------------------------------------------- the passes

def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "logprobs":
        return _logprobs(state, state["hidden"].detach().float(), state["weight"].detach().float())
    if state["op"] == "int8":
        q, sx = _quantize(state["hidden"])
        return _logprobs(state, q.float(), state["weight"].float(), sx[:, None] * state["weight_scale"])
    return _preference(state) if state["op"] == "preference" else _policy(state)


def _logprobs(s, x, w, product_scale=None):
    t, cap, scale = s["targets"], s["cap"], s["scale"]
    z = x @ w.t()
    if product_scale is not None:
        z = z * product_scale
    if s["bias"] is not None:
        z = z + s["bias"].detach().float()
    z = z * scale
    if cap:
        z = cap * torch.tanh(z / cap)
    valid = t != -100
    at = torch.where(valid, t, torch.zeros_like(t))[:, None]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lp = z - m - torch.log(total)
    p = e / total
    ent = -(p * lp).sum(1)
    out = dict(logps=torch.where(valid, lp.gather(1, at)[:, 0], 0.0), entropy=torch.where(valid, ent, 0.0))
    if not s.get("back"):
        return out
    g = torch.where(valid, s["grad_logps"], 0.0)[:, None]
    ge = torch.where(valid, s["grad_entropy"], 0.0)[:, None]
    d = -p * (g + ge * (lp + ent[:, None]))
    d.scatter_add_(1, at, g)
    if cap:
        d = d * (1 - (z / cap) ** 2)
    d = d * scale
    dt = s["hidden"].dtype
    out["grad_hidden"] = (d @ w).to(dt)
    out["grad_weight"] = (d.t() @ x).to(dt)
    if s["bias"] is not None:
        out["grad_bias"] = d.sum(0).to(dt)
    return out


def _per_token(s, y):
    """A value of each sequence at each of its tokens."""
    if s["offsets"] is None:
        return y[:, None].expand(s["logps"].shape)
    at = torch.arange(s["logps"].shape[0], device=y.device)
    return y[(torch.searchsorted(s["offsets"], at, right=True) - 1).clamp(max=s["seqs"] - 1)]


def _per_sequence(s, x):
    """Sums over each sequence, of thousands of terms: in 64 bits."""
    if s["offsets"] is None:
        return x.double().sum(1)
    edges = torch.cat([torch.zeros(1, dtype=torch.float64, device=x.device), x.double().cumsum(0)])[s["offsets"]]
    return edges[1:] - edges[:-1]


def _kept(s):
    if s["offsets"] is None:
        return s["mask"]
    return torch.arange(s["logps"].shape[0], device=s["logps"].device) < s["offsets"][-1]


def _preference(s):
    lp = s["logps"].detach().float()
    keep = _kept(s)
    count = _per_sequence(s, keep)
    ratio = lp if s["ref_logps"] is None else lp - s["ref_logps"].float()
    sums = _per_sequence(s, torch.where(keep, ratio, 0.0))
    per = 1 / count.clamp_min(1) if s["normalize"] else torch.ones_like(count)
    rewards = BETA * sums * per
    pairs = s["seqs"] // 2
    h = rewards[:pairs] - rewards[pairs:]
    if s["loss"] == "sigmoid":
        eps = s["smoothing"]
        soft = torch.clamp(-h, min=0) + torch.log1p(torch.exp(-torch.abs(h)))     # -log sigmoid(h)
        loss = (1 - eps) * soft + eps * (soft + h)
        slope = 1 / (1 + torch.exp(-h)) - (1 - eps)
    elif s["loss"] == "hinge":
        loss = torch.clamp(1 - h, min=0)
        slope = -(h < 1).double()
    else:
        loss = (h / BETA - 1 / (2 * BETA)) ** 2
        slope = 2 * (h / BETA - 1 / (2 * BETA)) / BETA
    coef = torch.cat([slope, -slope]) * BETA * per / pairs
    grad = torch.where(keep, _per_token(s, coef), 0.0).to(s["logps"].dtype)
    return dict(loss=loss.mean().float(), chosen=rewards[:pairs].float(), rejected=rewards[pairs:].float(), grad=grad)


CLIP_LOW, CLIP_HIGH, DUAL, KL, ENTROPY = 0.2, 0.28, 3.0, 0.05, 0.01


def _policy(s):
    dt = s["logps"].dtype
    lp, old = s["logps"].detach().float(), s["old_logps"].float()
    keep = _kept(s)
    count = _per_sequence(s, keep)
    adv = _per_token(s, s["advantages"]) if s["per_sequence"] else s["advantages"]
    x = lp.double() - old.double()                        # on which side of a clipping border a ratio lies: 64 bits
    r = torch.exp(x.float())
    low, high = r.new_tensor(1 - CLIP_LOW), r.new_tensor(1 + CLIP_HIGH)
    active = torch.where(adv < 0, x >= math.log(1 - CLIP_LOW), x <= math.log(1 + CLIP_HIGH))
    plain = r * adv
    gain = torch.where(active, plain, torch.where(adv < 0, low, high) * adv)
    if s["dual"]:
        bounded = (adv < 0) & (x > math.log(DUAL))
        gain = torch.where(bounded, DUAL * adv, gain)
        active = active & ~bounded
    loss = -gain
    d = -torch.where(active, plain, 0.0)
    if s["ref_logps"] is not None:
        away = (s["ref_logps"].float() - lp).double()        # e^x - x - 1 near 0
        loss = loss + KL * (torch.expm1(away) - away).float()
        d = d - KL * torch.expm1(away).float()
    if s["entropies"] is not None:
        loss = loss - ENTROPY * s["entropies"].detach().float()
    loss = torch.where(keep, loss, 0.0)
    d = torch.where(keep, d, 0.0)
    weight = keep.float()
    if s["reduction"] == "mean":
        weight = weight / count.sum().float()
    elif s["reduction"] == "sequence_mean":
        per = (1 / (count.clamp_min(1) * (count > 0).sum())).float()
        weight = weight * _per_token(s, per)
    weight = weight * s["grad"]
    if s["reduction"] == "none":
        out = dict(loss=loss)
    elif s["reduction"] == "sum":
        out = dict(loss=loss.double().sum().float())
    else:
        out = dict(loss=(loss.double() * weight).sum().float())
    out["grad"] = (d * weight).to(dt)
    if s["entropies"] is not None:
        out["grad_entropy"] = (-ENTROPY * weight).to(dt)
    return out


def _run_own(s):
    import linear_cross_entropy_tiled_amd as flce
    if s["op"] in ("logprobs", "int8"):
        opts = dict(logit_scale=s["scale"], softcap=s["cap"] or None, return_entropy=True)
        if s["op"] == "int8":
            lp, ent = flce.token_logprobs_int8(s["hidden"], s["weight"], s["weight_scale"], s["targets"], s["bias"],
                                               **opts)
        else:
            lp, ent = flce.token_logprobs(s["hidden"], s["weight"], s["targets"], s["bias"], **opts)
        out = dict(logps=lp.detach(), entropy=ent.detach())
        if s.get("back"):
            leaves = [s[k] for k in ("hidden", "weight", "bias") if s[k] is not None]
            grads = torch.autograd.grad((lp, ent), leaves, (s["grad_logps"], s["grad_entropy"]))
            out.update(zip(("grad_hidden", "grad_weight", "grad_bias"), grads))
        return out
    ref = s["ref_logps"].detach() if s["reference"] else None         # constants of both losses
    if s["op"] == "preference":
        loss, metrics = flce.preference_loss(s["logps"], ref, offsets=s["offsets"], mask=s["mask"],
                                             beta=BETA, loss_type=s["loss"], label_smoothing=s["smoothing"],
                                             length_normalize=s["normalize"], return_metrics=True)
        grad, = torch.autograd.grad(loss, (s["logps"],))
        return dict(loss=loss.detach(), chosen=metrics["chosen_rewards"], rejected=metrics["rejected_rewards"],
                    grad=grad)
    loss = flce.policy_loss(s["logps"], s["old_logps"].detach(), s["advantages"], ref_logps=ref,
                            entropy=s["entropies"], offsets=s["offsets"], mask=s["mask"], clip_low=CLIP_LOW,
                            clip_high=CLIP_HIGH, dual_clip=DUAL if s["dual"] else None,
                            kl_coef=KL if s["reference"] else 0.0, entropy_coef=ENTROPY if s["entropy"] else 0.0,
                            reduction=s["reduction"], advantages_per_sequence=s["per_sequence"])
    leaves = (s["logps"],) if s["entropies"] is None else (s["logps"], s["entropies"])
    grads = torch.autograd.grad(loss, leaves, s["grad"])
    out = dict(loss=loss.detach(), grad=grads[0])
    if s["entropies"] is not None:
        out["grad_entropy"] = grads[1]
    return out


# ----------------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("logprobs", "int8"):
        return _exact_logprobs(s)
    b = case["seqs"]
    lp = s["logps"].detach().double()
    if case["packed"]:
        sizes = s["offsets"][1:] - s["offsets"][:-1]
        kept = torch.zeros(lp.shape[0], dtype=torch.bool, device="cuda")
        kept[:int(s["offsets"][-1])] = True
        seq = torch.zeros(lp.shape[0], dtype=torch.int64, device="cuda")
        seq[kept] = torch.repeat_interleave(torch.arange(b, device="cuda"), sizes)
        group = lambda x: torch.zeros(b, dtype=torch.float64, device="cuda").scatter_add_(0, seq, x * kept)  # noqa: E731
        spread = lambda y: y[seq]  # noqa: E731
    else:
        kept = s["mask"]
        group = lambda x: x.sum(1)  # noqa: E731
        spread = lambda y: y[:, None].expand(lp.shape)  # noqa: E731
    n = group(kept.double())
    ref = s["ref_logps"].double() if s["ref_logps"] is not None else None
    if case["op"] == "preference":
        log_ratio = group(torch.where(kept, lp - (0 if ref is None else ref), 0.0))
        each = 1 / n.clamp_min(1) if case["normalize"] else torch.ones_like(n)
        reward = 0.1 * log_ratio * each
        half = b // 2
        h = (reward[:half] - reward[half:]).requires_grad_(True)
        ls = torch.nn.functional.logsigmoid
        if case["loss"] == "sigmoid":
            value = -(1 - case["smoothing"]) * ls(h) - case["smoothing"] * ls(-h)
        elif case["loss"] == "hinge":
            value = torch.relu(1 - h)
        else:
            value = (10 * h - 5) ** 2
        value = value.mean()
        dh, = torch.autograd.grad(value, h)
        to = torch.cat([dh, -dh]) * 0.1 * each
        return dict(loss=value.detach(), chosen=reward[:half], rejected=reward[half:],
                    grad=torch.where(kept, spread(to), 0.0))
    lp.requires_grad_(True)
    adv = spread(s["advantages"].double()) if case["per_sequence"] else s["advantages"].double()
    r = torch.exp(lp - s["old_logps"].double())
    gain = torch.minimum(r * adv, r.clamp(0.8, 1.28) * adv)
    if case["dual"]:
        gain = torch.where(adv < 0, torch.maximum(gain, 3.0 * adv), gain)
    value = -gain
    if ref is not None:
        value = value + 0.05 * (torch.expm1(ref - lp) - (ref - lp))
    at = (lp,)
    if case["entropy"]:
        ent = s["entropies"].detach().double().requires_grad_(True)
        value = value - 0.01 * ent
        at = (lp, ent)
    value = torch.where(kept, value, 0.0)
    if case["reduction"] == "mean":
        value = value.sum() / n.sum()
    elif case["reduction"] == "sequence_mean":
        value = (group(value) / n.clamp_min(1)).sum() / (n > 0).sum()
    elif case["reduction"] == "sum":
        value = value.sum()
    grads = torch.autograd.grad(value, at, s["grad"].double())
    out = dict(loss=value.detach(), grad=grads[0])
    if case["entropy"]:
        out["grad_entropy"] = grads[1]
    return out


def _exact_logprobs(s):
    x, t, cap, scale = s["hidden"].detach(), s["targets"], s["cap"], s["scale"]
    if s["op"] == "int8":
        q, sx = _quantize(x)          # the 8-bit values are defined by 32-bit operations
        x = q.double() * sx.double()[:, None]
        w = s["weight"].double() * s["weight_scale"].double()[:, None]
    else:
        x, w = x.double(), s["weight"].detach().double()
    bias = s["bias"].detach().double() if s["bias"] is not None else 0.0
    n, back = x.shape[0], bool(s.get("back"))
    logps = torch.zeros(n, dtype=torch.float64, device="cuda")
    ent = torch.zeros_like(logps)
    gx, gw = torch.zeros_like(x) if back else None, torch.zeros_like(w) if back else None
    gb = torch.zeros(w.shape[0], dtype=torch.float64, device="cuda")
    for i in range(0, n, 1024):
        rows = slice(i, min(i + 1024, n))
        u = scale * (x[rows] @ w.t() + bias)
        z = cap * torch.tanh(u / cap) if cap else u
        lp = torch.log_softmax(z, 1)
        live = (t[rows] != -100).double()
        hot = torch.zeros_like(lp).scatter_(1, t[rows].clamp_min(0)[:, None], live[:, None])
        logps[rows] = (hot * lp).sum(1)
        p = lp.exp()
        hh = -(p * lp).sum(1)
        ent[rows] = live * hh
        if back:
            g = (live * s["grad_logps"].double()[rows])[:, None]
            ge = (live * s["grad_entropy"].double()[rows])[:, None]
            d = g * (hot - p) - ge * p * (lp + hh[:, None])
            d = d * scale * ((1 - torch.tanh(u / cap) ** 2) if cap else 1.0)
            gx[rows] = d @ w
            gw += d.t() @ x[rows]
            gb += d.sum(0)
    out = dict(logps=logps, entropy=ent)
    if back:
        out.update(grad_hidden=gx, grad_weight=gw)
        if s["bias"] is not None:
            out["grad_bias"] = gb
    return out
