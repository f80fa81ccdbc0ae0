"""Autograd records none of the experts' calls: tensors that require a gradient
are refused while it is on, and never quietly cut off."""

import os

import pytest
import torch

import dimuon_newton_schulz_amd as D
from test_experts import announce, rows_of, weight

gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built")


class Calls:
    """Tensors of every call, on one device."""

    def __init__(self, device):
        def rows(n, width, seed):
            return torch.randn(n, width, generator=torch.Generator().manual_seed(seed)).to(device)

        ids = torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=torch.int32, device=device)
        self.routes = D.expert_sort(ids, 2) if device == "cuda" else \
            D.ExpertRoutes(torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), ids)
        self.t = {"x": rows(3, 8, 1), "xs": rows(6, 8, 2), "weights": rows(3, 2, 3), "residual": rows(3, 8, 4), "w": rows(4, 8, 5),
                  "bias": rows(1, 4, 6)[0], "res": rows(3, 4, 7), "out": rows(3, 4, 8), "pre": rows(3, 4, 9), "y": rows(3, 8, 10),
                  "dy": rows(3, 4, 11), "dx": rows(3, 8, 12)}

    def all(self):
        t, r = self.t, self.routes
        return {
            "gather": (("x",), lambda: D.expert_gather(t["x"], r)),
            "gather_out": (("x", "xs"), lambda: D.expert_gather(t["x"], r, out=t["xs"])),
            "combine": (("xs", "weights", "residual", "y"),
                        lambda: D.expert_combine(t["xs"], r, t["weights"], t["residual"], t["y"])),
            "combine_grad": (("x",), lambda: D.expert_combine_grad(t["x"], t["xs"], t["weights"], r)),
            "linear": (("x", "w", "bias", "res", "out", "pre"),
                       lambda: D.linear(t["x"], t["w"], t["bias"], "silu", t["res"], None, t["pre"], t["out"])),
            "linear_grad": (("dy",), lambda: D.linear_grad(t["dy"], w=t["w"], dx=t["dx"])),
        }


def refused(calls):
    for call, (names, run) in calls.all().items():
        for name in names:
            calls.t[name].requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                run()
            calls.t[name].requires_grad_(False)


@built
def test_tensors_that_require_a_gradient_are_refused():
    refused(Calls("cpu"))


@gpu
def test_tensors_that_require_a_gradient_are_refused_on_the_gpu():
    announce("tensors that require a gradient")
    calls = Calls("cuda")
    refused(calls)
    for call, (names, run) in calls.all().items():   # and taken while autograd is off
        want = run()
        for name in names:
            calls.t[name].requires_grad_()
        with torch.no_grad():
            got = run()
        for name in names:
            calls.t[name].requires_grad_(False)
        for a, b in zip(*((v,) if isinstance(v, torch.Tensor) else v for v in (want, got))):
            assert (a is None and b is None) or (torch.equal(a, b) and not (b.requires_grad and b.grad_fn)), call


@gpu
def test_weights_that_require_a_gradient_in_a_backward_of_ones_own():
    """A parameter in linear_grad, whose gradient goes into its .grad."""
    announce("a parameter's own gradient buffer")
    p = torch.nn.Parameter(rows_of(4, 8, torch.float32, 1))
    x, dy = rows_of(10, 8, torch.float32, 2), rows_of(10, 4, torch.float32, 3)
    p.grad = torch.zeros_like(p)
    dx = torch.empty_like(x)
    D.linear_grad(dy, x, p, dx=dx, dw=p.grad)
    assert torch.allclose(p.grad, dy.t() @ x, atol=1e-4) and torch.allclose(dx, dy @ p.detach(), atol=1e-4)


@gpu
def test_function_of_ones_own():
    """The calls in a torch.autograd.Function give autograd's gradients."""
    announce("autograd.Function")

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            pre = torch.empty(len(x), len(w), device="cuda")
            ctx.save_for_backward(x, w, pre)
            return D.linear(x, w, activation="silu", pre=pre)

        @staticmethod
        def backward(ctx, dy):
            x, w, pre = ctx.saved_tensors
            return D.linear_grad(dy.contiguous(), x, w, activation="silu", pre=pre, dx=torch.empty_like(x),
                                 dw=torch.empty_like(w))[:2]

    x, w = rows_of(30, 16, torch.float32, 1).requires_grad_(), weight(1, 12, 16, torch.float32, 2)[0].clone().requires_grad_()
    got = torch.autograd.grad(Linear.apply(x, w).square().sum(), (x, w))
    want = torch.autograd.grad(torch.nn.functional.silu(x.double() @ w.double().t()).square().sum(), (x, w))
    # sums of up to 30 products in float32, of values of order one: 1e-5 of the largest
    for a, b in zip(got, want):
        assert (a - b).abs().max() < 1e-5 * b.abs().max() + 1e-6
