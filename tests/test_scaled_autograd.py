"""The differentiable linear layer as autograd sees it.  On the CPU the quantiser
and the product stand in as plain torch (what is tested is which of them are
called, and what is kept); on the GPU they are the kernels."""
import pytest
import torch

import exact_integer_gemm_amd as rg
from exact_integer_gemm_amd import scaled

M, N, K = 5, 7, 6


class Stand:
    """Stand-ins that keep entries as they are, with scales of one, and count calls."""

    def __init__(self):
        self.calls = []

    def block_quantize(self, x, dtype=None, block_rows=1, scale_dtype=torch.float32):
        self.calls.append("one")
        return x.detach().clone(), torch.ones(1, 1, dtype=scale_dtype)

    def block_quantize_both(self, x, dtype=None, block_rows=1, scale_dtype=torch.float32):
        self.calls.append("both")
        one = torch.ones(1, 1, dtype=scale_dtype)
        return x.detach().clone(), one, x.detach().t().contiguous(), one.clone()

    def scaled_mm_nt(self, a, a_scales, b, b_scales, out_dtype=torch.bfloat16, out=None, workspace=None):
        self.calls.append("mm")
        return (a @ b.t()).to(out_dtype)


@pytest.fixture(params=["stand", pytest.param("gpu", marks=pytest.mark.gpu)])
def layer(request, monkeypatch):
    """(device, the stand-ins or None)."""
    if request.param == "gpu":
        return "cuda", None
    stand = Stand()
    for name in ("block_quantize", "block_quantize_both", "scaled_mm_nt"):
        monkeypatch.setattr(scaled, name, getattr(stand, name))
    return "cpu", stand


def operands(device, x_grad=True, w_grad=True):
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((M, K), generator=g).to(device), torch.randn((N, K), generator=g).to(device)
    return x.requires_grad_(x_grad), w.requires_grad_(w_grad)


def run(x, w):
    return rg.scaled_linear(x, w, scale_dtype=torch.float32)


def test_gradients_reach_both_operands(layer):
    device, stand = layer
    x, w = operands(device)
    dy = torch.randn((M, N), generator=torch.Generator().manual_seed(2)).to(device)
    run(x, w).backward(dy)
    # the kernels' operands are off by at most half a step of e4m3, 2^-4, each
    tol = 1e-6 if stand else 2 * 2.0 ** -4 + 2.0 ** -8
    for got, want, size in ((x.grad, dy @ w, dy.abs() @ w.abs()), (w.grad, dy.t() @ x, dy.abs().t() @ x.abs())):
        assert bool(((got - want).abs() <= tol * size + 1e-6).all())


def test_second_derivatives_are_refused(layer):
    """A gradient penalty would lose its term without a word."""
    device, _ = layer
    x, w = operands(device)
    gx, = torch.autograd.grad(run(x, w).square().sum(), x, create_graph=True)
    penalty = gx.square().sum() + (w * w).sum()
    with pytest.raises(RuntimeError, match="twice|once_differentiable"):
        penalty.backward()


def test_what_is_kept_goes_through_the_graph(layer):
    """Hooks on saved tensors (offloading, checkpointing) see it, and a backward pass frees it."""
    device, _ = layer
    x, w = operands(device)
    seen = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t.shape) or t, lambda t: t):
        y = run(x, w)
    assert sum(s[0] == K and s[1] >= M for s in seen) == 2       # x and the weight, transposed
    y.sum().backward()
    with pytest.raises(RuntimeError, match="second time"):
        y.sum().backward()
    x.grad = w.grad = None
    y = run(x, w)
    y.sum().backward(retain_graph=True)
    first = x.grad.clone(), w.grad.clone()
    y.sum().backward()
    assert torch.equal(x.grad, 2 * first[0]) and torch.equal(w.grad, 2 * first[1])


@pytest.mark.gpu
def test_what_is_kept_may_leave_the_device():
    """Kept on the host until it is needed, to the same bits."""
    g = torch.Generator().manual_seed(3)
    x, w, dy = (torch.randn(s, generator=g).cuda() for s in ((70, 200), (90, 200), (70, 90)))
    x.requires_grad_(), w.requires_grad_()
    run(x, w).backward(dy)
    here = x.grad, w.grad
    x.grad = w.grad = None
    with torch.autograd.graph.save_on_cpu():
        y = run(x, w)
    y.backward(dy)
    assert torch.equal(x.grad, here[0]) and torch.equal(w.grad, here[1])


def test_recomputed_layers(layer):
    """Non-reentrant checkpointing gives the gradients of the plain pass."""
    from torch.utils.checkpoint import checkpoint
    device, _ = layer
    grads = []
    for again in (False, True):
        x, w = operands(device)
        y = checkpoint(run, x, w, use_reentrant=False) if again else run(x, w)
        y.square().sum().backward()
        grads.append((x.grad, w.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


@pytest.mark.parametrize("x_grad,w_grad,grad_mode,forward,backward", [
    (True, True, True, ["both", "both", "mm"], ["both", "mm", "mm"]),
    (True, False, True, ["one", "both", "mm"], ["one", "mm"]),         # a frozen weight: dy along N, the weight transposed
    (False, True, True, ["both", "one", "mm"], ["both", "mm"]),        # the first layer
    (False, False, True, ["one", "one", "mm"], None),
    (True, True, False, ["one", "one", "mm"], None),                   # inference
])
def test_only_what_the_gradients_need_is_quantised(layer, x_grad, w_grad, grad_mode, forward, backward):
    device, stand = layer
    x, w = operands(device)
    want = run(x, w)
    want.square().sum().backward()
    gx, gw = x.grad, w.grad
    x, w = operands(device, x_grad, w_grad)
    if stand:
        stand.calls.clear()
    with torch.set_grad_enabled(grad_mode):
        y = run(x, w)
    assert torch.equal(y, want) and y.requires_grad == (backward is not None)
    if stand:
        assert stand.calls == forward
        stand.calls.clear()
    if backward is None:
        return
    y.square().sum().backward()
    assert (x.grad is None) == (not x_grad) and (w.grad is None) == (not w_grad)
    assert (x.grad is None or torch.equal(x.grad, gx)) and (w.grad is None or torch.equal(w.grad, gw))
    assert stand is None or stand.calls == backward


def test_other_modes_are_refused(layer):
    device, _ = layer
    x, w = operands(device, False, False)
    with torch.autograd.forward_ad.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        run(torch.autograd.forward_ad.make_dual(x, torch.ones_like(x)), w)
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.vmap(lambda t: run(t, w))(x.unsqueeze(0))
