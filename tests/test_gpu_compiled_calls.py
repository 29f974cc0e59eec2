"""torch.compile of a function that calls the package: its functions run between the compiled pieces, with the
results, gradients and refusals of the eager call, bit for bit (the pieces here only negate and double, which is exact)."""
import pytest

pytestmark = pytest.mark.gpu
BACKENDS = ["eager", "aot_eager"]
N, H, V = 33, 96, 300


def _made(seed=0):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(N, H, device="cuda", generator=g)
    w, b = torch.randn(H, device="cuda", generator=g), torch.randn(H, device="cuda", generator=g)
    head = torch.randn(V, H, device="cuda", generator=g)
    ids = torch.randint(0, V, (N,), device="cuda", generator=g)
    return x, w, b, head, ids


def _same(fn, args, backend):
    """fn compiled against fn, values and the gradients of its floating arguments."""
    import torch
    torch._dynamo.reset()
    compiled = torch.compile(fn, backend=backend)
    for _ in range(2):                                   # traced, then run again
        out = []
        for f in (fn, compiled):
            leaves = [a.clone().requires_grad_(True) if a.is_floating_point() else a for a in args]
            y = f(*leaves)
            y = y if isinstance(y, tuple) else (y,)
            recorded = [t for t in y if t.requires_grad]
            grads = []
            if recorded:
                ups = [torch.linspace(-1, 1, t.numel(), device="cuda").view_as(t).to(t.dtype) for t in recorded]
                grads = list(torch.autograd.grad(recorded, [a for a in leaves if a.requires_grad], ups))
            out.append([t.detach() for t in y] + grads)
        assert len(out[0]) == len(out[1]) and all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("backend", BACKENDS)
def test_layer_norm(flce_lib, backend):
    x, w, b, _, _ = _made()
    _same(lambda x, w, b: flce_lib.layer_norm(-x, w, b, eps=1e-3) * 2, (x, w, b), backend)
    _same(lambda x: flce_lib.layer_norm(-x) * 2, (x,), backend)


@pytest.mark.parametrize("backend", BACKENDS)
def test_embedding(flce_lib, backend):
    *_, head, ids = _made()
    _same(lambda head, ids: -flce_lib.embedding(ids, head * 2, scale=3.0), (head, ids), backend)


@pytest.mark.parametrize("backend", BACKENDS)
def test_embedding_backward(flce_lib, backend):
    import torch
    x, _, _, _, ids = _made()

    def fn(ids):
        return -flce_lib.embedding_backward(x * 2, ids, V)

    _same(fn, (ids,), backend)
    buffer = torch.ones(V, H, device="cuda")
    torch._dynamo.reset()
    got = torch.compile(lambda: flce_lib.embedding_backward(x, ids, V, grad_weight=buffer), backend=backend)()
    assert got is buffer and torch.equal(buffer, flce_lib.embedding_backward(x, ids, V, grad_weight=torch.ones_like(buffer)))


@pytest.mark.parametrize("backend", BACKENDS)
def test_mxfp4(flce_lib, backend):
    import torch
    x, _, _, head, ids = _made()

    def fn(ids):
        q, s = flce_lib.quantize_mxfp4(head * 2)
        logps, entropy = flce_lib.token_logprobs_mxfp4(-x, q, s, ids, return_entropy=True)
        xq, xs = flce_lib.quantize_mxfp4(-x)
        codes = flce_lib.token_logprobs_mxfp4(xq, q, s, ids, hidden_scale=xs, softcap=5.0)
        return q, s, flce_lib.dequantize_mxfp4(q, s, torch.bfloat16) * 2, -logps, -entropy, -codes

    _same(fn, (ids,), backend)


def _losses(flce_lib):
    """name -> (function, its arguments)."""
    import torch
    x, _, _, head, ids = _made()
    x, head = (x * 0.3).bfloat16(), (head * 0.3).bfloat16()
    lp = -torch.rand(4, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    one, adv = torch.ones(1, device="cuda"), torch.linspace(-1, 1, 4, device="cuda")
    lse = flce_lib.forward(x, head, ids, reduction="mean")[1]
    q, s = flce_lib.quantize_int8(head)
    target = torch.zeros(N, V, device="cuda")
    rows, columns = torch.ones(N, device="cuda"), torch.ones(V, device="cuda")

    def policy(lp):
        return flce_lib.policy_loss(lp * 2, lp.detach(), adv)

    def preference(lp):
        return flce_lib.preference_loss(lp * 2, lp.detach())

    return {
        "forward": (lambda x: flce_lib.forward(-x, head, ids, reduction="mean")[:2], (x,)),
        "backward": (lambda x: flce_lib.backward(-x, head, ids, lse, one, reduction="mean")[:2], (x,)),
        "forward_backward": (lambda x: flce_lib.forward_backward(-x, head, ids, one, reduction="mean")[0], (x,)),
        "linear_cross_entropy": (lambda x, w: flce_lib.linear_cross_entropy(-x, w, ids, reduction="mean") * 2, (x, head)),
        "weighted_mse": (lambda x: flce_lib.weighted_mse(-x, head, target, rows, columns)[0], (x,)),
        "token_logprobs": (lambda x, w: -flce_lib.token_logprobs(-x, w, ids), (x, head)),
        "quantize_int8": (lambda x: flce_lib.quantize_int8(-x), (x,)),
        "token_logprobs_int8": (lambda ids: -flce_lib.token_logprobs_int8(-x, q, s, ids), (ids,)),
        "policy_loss": (policy, (lp,)),
        "preference_loss": (preference, (lp,)),
    }


@pytest.mark.parametrize("backend", BACKENDS)
@pytest.mark.parametrize("name", ["forward", "backward", "forward_backward", "linear_cross_entropy", "weighted_mse",
                                  "token_logprobs", "quantize_int8", "token_logprobs_int8", "policy_loss",
                                  "preference_loss"])
def test_losses_and_scores(flce_lib, name, backend):
    _same(*_losses(flce_lib)[name], backend)


@pytest.mark.parametrize("backend", BACKENDS)
def test_refusals_come_through(flce_lib, backend):
    import torch
    x, w, b, head, ids = _made()
    torch._dynamo.reset()
    with pytest.raises(ValueError):
        torch.compile(lambda x: flce_lib.layer_norm(-x, w[1:], b), backend=backend)(x)
    with pytest.raises(TypeError):
        torch.compile(lambda i: flce_lib.embedding(i.float(), head), backend=backend)(ids)


def test_one_whole_graph_is_refused(flce_lib):
    import torch
    x, w, b, _, _ = _made()
    torch._dynamo.reset()
    with pytest.raises(torch._dynamo.exc.Unsupported):
        torch.compile(lambda x: flce_lib.layer_norm(-x, w, b), backend="eager", fullgraph=True)(x)
