"""Operators at the ends of a language model as measurable cases: token embedding with its gradient, layer norm with
its gradients, 4-bit microscaled (MXFP4) quantisation, and log-probabilities of a frozen MXFP4 head.

``own`` false: the operators in elementary torch operations.  ``own`` true: the framework's entry points."""
import math

import torch

own = False

SHARE_PADDED = 0.05          # tokens without an id, rows whose target is ignored
EPS = 1e-5


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch
        dict(name="embedding lookup n16", op="embedding", dtype="bf16", n=16, h=4096, v=32000, scale=1.0, back=False),
        # a debugging run in single precision: odd sizes, rows that are not aligned, embeddings scaled by sqrt(h)
        dict(name="embedding train f32", op="embedding", dtype="f32", n=2001, h=1023, v=8191, scale=31.984371,
             back=True),
        # the training step of a model with a large vocabulary
        dict(name="embedding train bf16", op="embedding", dtype="bf16", n=8192, h=4096, v=128256, scale=1.0,
             back=True),
        # the last norm before the head in one decoding step
        dict(name="layer norm n16", op="norm", dtype="bf16", params="bf16", n=16, h=4096, bias=True, back=False),
        # single precision, odd sizes
        dict(name="layer norm train f32", op="norm", dtype="f32", params="f32", n=515, h=1023, bias=True, back=True),
        # a training step in 16 bits whose parameters are kept in 32
        dict(name="layer norm train bf16", op="norm", dtype="bf16", params="f32", n=8192, h=4096, bias=True,
             back=True),
        # a long batch in half precision, no bias
        dict(name="layer norm train f16", op="norm", dtype="f16", params="f16", n=65536, h=2048, bias=False,
             back=True),
        # the hidden states of one answer as a user inspects them: what 4 bits keep of each
        dict(name="mxfp4 values n250", op="quantize", dtype="bf16", n=250, h=4096),
        # a head as it is laid out when a scorer is loaded, and read back
        dict(name="mxfp4 values head", op="quantize", dtype="bf16", n=128256, h=4096),
        # a frozen scorer's 4-bit head: the tokens of one decoding step
        dict(name="mxfp4 score n4", op="score", dtype="bf16", n=4, h=4096, v=128256, bias=False, scale=1.0, cap=0.0),
        # one ragged packed answer batch, capped logits and a bias
        dict(name="mxfp4 score n1000", op="score", dtype="f16", n=1000, h=2048, v=50001, bias=True, scale=1.0,
             cap=30.0),
        # the reference's scores of a whole training batch
        dict(name="mxfp4 score n8192", op="score", dtype="bf16", n=8192, h=4096, v=128256, bias=False, scale=1.0,
             cap=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "norm", "quantize", "score"])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32", "bf16"]))
    if op == "embedding":
        case.update(n=_log_int(rng, 1, 32768), h=_log_int(rng, 64, 4096), v=_log_int(rng, 500, 128256),
                    scale=rng.choice([1.0, 1.0, 22.627417]), back=rng.random() < 0.7)
        if rng.random() < 0.6:
            case["h"] = (case["h"] + 7) // 8 * 8
        if case["dtype"] == "f32":
            case["v"] = min(case["v"], 64128)
    elif op == "norm":
        case.update(params=rng.choice(["f32", case["dtype"]]), n=_log_int(rng, 1, 65536), h=_log_int(rng, 64, 8192),
                    bias=rng.random() < 0.5, back=rng.random() < 0.7)
        if rng.random() < 0.6:
            case["h"] = (case["h"] + 7) // 8 * 8
        case["n"] = max(1, min(case["n"], (1 << 26) // case["h"]))
    elif op == "quantize":
        case.update(n=_log_int(rng, 1, 128256), h=32 * _log_int(rng, 2, 128))
    else:
        case.update(n=_log_int(rng, 1, 8192), h=32 * _log_int(rng, 4, 128), v=_log_int(rng, 500, 128256),
                    bias=rng.random() < 0.4, scale=rng.choice([1.0, 0.7, 1.25]), cap=rng.choice([0.0, 0.0, 30.0]))
    return case


TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------------------- MXFP4, the plain form

# 32 neighbouring values share one power of two, 2^(code - 127); each is one of +-{0, .5, 1, 1.5, 2, 3, 4, 6} times it.
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_split(x):
    """(R, H) values: codes 0 .. 15 (R, H) and scale codes (R, H / 32).  The scale's exponent is that of the block's
    largest magnitude less 2, the grid's rounding is to the nearest, ties to the even code, past 6 it saturates.  A
    block with NaN or an infinity has scale code 255 (NaN) and codes 0."""
    r, h = x.shape
    b = x.float().view(r, h // 32, 32)
    top = b.abs().amax(2)
    _, e = torch.frexp(top)                               # top = m 2^e, m in [1/2, 1)
    e = torch.where(top > 0, e - 3, -127).clamp(-127, 127)
    finite = torch.isfinite(b).all(2)
    e = torch.where(finite, e, 0)
    y = torch.ldexp(b.abs(), -e[..., None])
    code = (y > 0.25).to(torch.uint8)
    for edge, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (y >= edge) if up else (y > edge)
    code += 8 * (b < 0).to(torch.uint8)
    code = torch.where(finite[..., None], code, 0)
    return code.view(r, h), torch.where(finite, e + 127, 255).to(torch.uint8)


def _mx_values(code, scale):
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float32, device=code.device)
    r, h = code.shape
    s = torch.ldexp(torch.ones((), device=code.device), scale.int() - 127)
    s = torch.where(scale == 255, float("nan"), s)
    return (grid[code.int()].view(r, h // 32, 32) * s[..., None]).view(r, h)


def _mx_quantize(x):
    """What the framework stores: two codes a byte, the earlier one in the low half."""
    code, scale = _mx_split(x)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def _mx_unpack(q, scale):
    code = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)
    return _mx_values(code, scale)


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case)
    n, h, dt = case["n"], case["h"], TORCH[case["dtype"]]
    unit = (256.0 if case["dtype"] == "f16" else 1.0)           # half precision trains with a loss scale
    if case["op"] == "embedding":
        # ids by Zipf's law: the most frequent token is every twelfth or so, most of the vocabulary does not occur
        v = case["v"]
        ids = (torch.exp(rand(n) * math.log(v + 1)).long() - 1).clamp(0, v - 1)
        if n > 1:
            ids = torch.where(rand(n) < SHARE_PADDED, torch.full_like(ids, -100), ids)
        s["ids"] = ids
        s["weight"] = torch.empty(v, h, device="cuda").normal_(0, 0.02, generator=g).to(dt)
        if case["back"]:
            s["weight"].requires_grad_(True)
            s["grad"] = (unit / n * randn(n, h)).to(dt)
    elif case["op"] == "norm":
        # rows of different sizes and means, and a few large columns, as hidden states have them
        x = randn(n, h) * torch.exp(0.5 * randn(n, 1)) + 0.3 * randn(n, 1)
        x[:, ::97] *= 8
        s["x"] = x.to(dt)
        s["weight"] = (1 + 0.2 * randn(h)).to(TORCH[case["params"]])
        s["bias"] = (0.2 * randn(h)).to(TORCH[case["params"]]) if case["bias"] else None
        if case["back"]:
            s["grad"] = (unit / math.sqrt(n) * randn(n, h)).to(dt)
            for k in ("x", "weight", "bias"):
                if s[k] is not None:
                    s[k].requires_grad_(True)
    elif case["op"] == "quantize":
        x = torch.empty(n, h, device="cuda").normal_(0, 1, generator=g) if n < 4096 else None
        if x is None:                                                       # a head
            x = torch.empty(n, h, device="cuda").normal_(0, 1 / math.sqrt(h), generator=g)
        else:
            x = x * torch.exp(0.5 * randn(n, 1))
            x[:, ::97] *= 8
        s["x"] = x.to(dt)
    else:
        v = case["v"]
        w = torch.empty(v, h, device="cuda").normal_(0, 1 / math.sqrt(h), generator=g)
        targets = torch.randint(0, v, (n,), generator=g, device="cuda")
        # each token's state leans towards its target's row by its own amount: some tokens are almost sure, some not
        lean = rand(n, 1) * 1.5 * math.log(v)
        x = randn(n, h) + lean * w[targets]
        if n > 1:
            targets = torch.where(rand(n) < SHARE_PADDED, torch.full_like(targets, -100), targets)
        s["hidden"], s["targets"] = x.to(dt), targets
        s["bias"] = 0.3 * randn(v) if case["bias"] else None
        # laid out once, when the scorer is loaded
        parts = [_mx_quantize(p) for p in w.split(8192)]
        s["weight"] = torch.cat([p[0] for p in parts])
        s["weight_scale"] = torch.cat([p[1] for p in parts])
    return s


BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    n, h, e = case["n"], case["h"], BYTES[case["dtype"]]
    if case["op"] == "embedding":
        back = n * h * e + case["v"] * h * e if case["back"] else 0
        return {"bytes": 8 * n + 2 * n * h * e + back, "flops": 2.0 * n * h}
    if case["op"] == "norm":
        params = (2 if case["bias"] else 1) * h * BYTES[case["params"]]
        if not case["back"]:
            return {"bytes": 2 * n * h * e + params, "flops": 8.0 * n * h}
        # x twice: the gradient comes when the output is gone
        return {"bytes": 5 * n * h * e + 3 * params, "flops": 20.0 * n * h}
    if case["op"] == "quantize":
        return {"bytes": int(n * h * (2 * e + 17 / 32)), "flops": 4.0 * n * h}
    v = case["v"]
    return {"bytes": int(n * h * e + v * h * 17 / 32 + 16 * n), "flops": 2.0 * n * h * v}


# ----------------------------------------------------------------------------- the passes

def run(state):
    if own:
        return _run_own(state)
    return {"embedding": _embedding, "norm": _norm, "quantize": _quantize, "score": _score}[state["op"]](state)


def _embedding(s):
    w, ids = s["weight"].detach(), s["ids"]
    known = ((ids >= 0) & (ids < s["v"]))[:, None]
    at = torch.where(known[:, 0], ids, torch.zeros_like(ids))
    out = dict(out=torch.where(known, w[at].float() * s["scale"], 0.0).to(w.dtype))
    if s["back"]:
        grad = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
        grad.index_add_(0, at, torch.where(known, s["grad"].float() * s["scale"], 0.0))
        out["grad_weight"] = grad.to(w.dtype)
    return out


def _norm(s):
    x, w = s["x"].detach().float(), s["weight"].detach().float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    xhat = c * rstd
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"].detach().float()
    out = dict(out=y.to(s["x"].dtype))
    if s["back"]:
        dy = s["grad"].float()
        d = dy * w
        dx = rstd * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
        out["grad_x"] = dx.to(s["x"].dtype)
        out["grad_weight"] = (dy * xhat).sum(0).to(s["weight"].dtype)
        if s["bias"] is not None:
            out["grad_bias"] = dy.sum(0).to(s["bias"].dtype)
    return out


def _quantize(s):
    return dict(values=_mx_values(*_mx_split(s["x"])).to(s["x"].dtype))


def _score(s):
    t, cap, scale = s["targets"], s["cap"], s["scale"]
    z = _mx_values(*_mx_split(s["hidden"])) @ _mx_unpack(s["weight"], s["weight_scale"]).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    z = z * scale
    if cap:
        z = cap * torch.tanh(z / cap)
    valid = t != -100
    at = torch.where(valid, t, torch.zeros_like(t))[:, None]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    lp = z - torch.log(total)
    ent = -(e / total * lp).sum(1)
    return dict(logps=torch.where(valid, lp.gather(1, at)[:, 0], 0.0), entropy=torch.where(valid, ent, 0.0))


def _run_own(s):
    import linear_cross_entropy_tiled_amd as flce
    if s["op"] == "embedding":
        y = flce.embedding(s["ids"], s["weight"], scale=s["scale"])
        if not s["back"]:
            return dict(out=y)
        grad, = torch.autograd.grad(y, (s["weight"],), (s["grad"],))
        return dict(out=y.detach(), grad_weight=grad)
    if s["op"] == "norm":
        y = flce.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        if not s["back"]:
            return dict(out=y)
        leaves = [s[k] for k in ("x", "weight", "bias") if s[k] is not None]
        grads = torch.autograd.grad(y, leaves, (s["grad"],))
        return dict(zip(("out", "grad_x", "grad_weight", "grad_bias"), (y.detach(), *grads)))
    if s["op"] == "quantize":
        q, scale = flce.quantize_mxfp4(s["x"])
        return dict(values=flce.dequantize_mxfp4(q, scale, dtype=s["x"].dtype))
    lp, ent = flce.token_logprobs_mxfp4(s["hidden"], s["weight"], s["weight_scale"], s["targets"], s["bias"],
                                        logit_scale=s["scale"], softcap=s["cap"] or None, return_entropy=True)
    return dict(logps=lp, entropy=ent)


# ----------------------------------------------------------------------------- in 64 bits, from the definitions

def _exact_mx(x):
    """The values that MXFP4 keeps of (R, H) finite ones."""
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    # the exponent field of a double
    e = ((top.view(torch.int64) >> 52) & 2047) - 1023 - 2
    unit = ((e.clamp(-127, 127) + 1023) << 52).view(torch.float64)
    y = b.abs() / unit
    # spacing 1/2 below 2, 1 up to 4, 2 up to 6; torch.round takes ties to the even multiple, as the codes are
    # even: 0, 1, 2 | 2, 4 | 4 (and 8, which saturates)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.minimum(torch.round(y / step) * step, torch.full_like(y, 6.0))
    return (torch.sign(b) * y * unit).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embedding":
        ids, w = s["ids"], s["weight"].detach()
        keep = torch.nonzero((ids >= 0) & (ids < case["v"]))[:, 0]
        out = torch.zeros(case["n"], case["h"], dtype=torch.float64, device=ids.device)
        out[keep] = w[ids[keep]].double() * case["scale"]
        if not case["back"]:
            return dict(out=out)
        grad = torch.zeros(w.shape, dtype=torch.float64, device=ids.device)
        grad.index_put_((ids[keep],), s["grad"][keep].double() * case["scale"], accumulate=True)
        return dict(out=out, grad_weight=grad)
    if case["op"] == "norm":
        x, w = s["x"].detach().double(), s["weight"].detach().double()
        h = case["h"]
        mean = x.sum(1, keepdim=True) / h
        var = ((x - mean) ** 2).sum(1, keepdim=True) / h
        xhat = (x - mean) / (var + EPS) ** 0.5
        y = xhat * w
        if s["bias"] is not None:
            y += s["bias"].detach().double()
        out = dict(out=y)
        if case["back"]:
            dy = s["grad"].double()
            dxhat = dy * w
            inner = h * dxhat - dxhat.sum(1, keepdim=True) - xhat * (dxhat * xhat).sum(1, keepdim=True)
            out["grad_x"] = inner / (h * (var + EPS) ** 0.5)
            out["grad_weight"] = (dy * xhat).sum(0)
            if s["bias"] is not None:
                out["grad_bias"] = dy.sum(0)
        return out
    if case["op"] == "quantize":
        return dict(values=torch.cat([_exact_mx(p) for p in s["x"].split(8192)]))
    low = (s["weight"] & 15).long()
    high = (s["weight"] >> 4).long()
    grid = torch.tensor(GRID, dtype=torch.float64, device=low.device)
    w = torch.empty(case["v"], case["h"], dtype=torch.float64, device=low.device)
    for first, code in ((0, low), (1, high)):
        w[:, first::2] = grid[code & 7] * (1 - 2 * (code >> 3)).double()
    w = w * torch.pow(2.0, s["weight_scale"].double() - 127).repeat_interleave(32, 1)
    logps, entropy = [], []
    for x, t in zip(s["hidden"].split(256), s["targets"].split(256)):
        z = _exact_mx(x) @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].double()
        z = z * case["scale"]
        if case["cap"]:
            z = case["cap"] * torch.tanh(z / case["cap"])
        lp = torch.log_softmax(z, 1)
        keep = t != -100
        logps.append(torch.where(keep, lp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0))
        entropy.append(torch.where(keep, -(lp.exp() * lp).sum(1), 0.0))
    return dict(logps=torch.cat(logps), entropy=torch.cat(entropy))
