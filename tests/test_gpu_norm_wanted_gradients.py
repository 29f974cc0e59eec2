"""layer_norm's backward forms the gradients that a call asks for, and no others: told by the memory that the call takes
at its peak, of which an unwanted gradient of x would be another 64 MiB and the column sums' workspace another 16."""
import pytest

pytestmark = pytest.mark.gpu
N = H = 4096


SUBSETS = ["x", "w", "b", "x w", "x b", "w b", "x w b"]


@pytest.mark.parametrize("given,wanted", [(g, s) for g in ("x w b", "x w", "x b", "x", "w b") for s in SUBSETS
                                          if set(s) <= set(g)])
def test_a_subset_of_the_gradients(flce_lib, given, wanted):
    import torch
    given, wanted = given.split(), wanted.split()
    gen = torch.Generator("cuda").manual_seed(0)
    made = {k: torch.randn((N, H) if k == "x" else (H,), device="cuda", generator=gen) for k in "xwb"}
    leaves = {k: made[k].requires_grad_(k in given) for k in "xwb"}
    absent = [k for k in "wb" if k not in given and "x" in given]     # (x alone is there without being recorded)
    y = flce_lib.layer_norm(leaves["x"], *(None if k in absent else leaves[k] for k in "wb"))
    g = torch.randn(N, H, device="cuda", generator=gen)
    every = dict(zip(given, torch.autograd.grad(y, [leaves[k] for k in given], g, retain_graph=True)))
    p = flce_lib.flce_norm_params(N, H, 0, 0, 0, 0, 1e-5, 0)
    workspace = flce_lib.flce_layer_norm_workspace_size(p)
    need = sum(made[k].numel() * 4 for k in wanted) + (workspace if set(wanted) & {"w", "b"} else 0)
    assert workspace >= 1 << 24
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = torch.autograd.grad(y, [leaves[k] for k in wanted], g)
    taken = torch.cuda.max_memory_allocated() - before
    assert all(torch.equal(v, every[k]) for k, v in zip(wanted, got))
    assert taken < need + (1 << 22), (taken, need)       # 4 MiB: the allocator's rounding


def test_backward_into_some_leaves(flce_lib):
    import torch
    x, w, b = (torch.randn(*s, device="cuda", requires_grad=True) for s in ((33, 72), (72,), (72,)))
    y = flce_lib.layer_norm(x, w, b)
    want = torch.autograd.grad(y.sum(), (x, w, b), retain_graph=True)
    y.sum().backward(inputs=[b])
    assert x.grad is None and w.grad is None and torch.equal(b.grad, want[2])
    flce_lib.layer_norm(x, w, b).sum().backward()
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1]) and torch.equal(b.grad, 2 * want[2])
