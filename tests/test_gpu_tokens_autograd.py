"""The token path under autograd: inside autograd.Functions it gives the gradients of its own entry points; outside of
them tensors that require a gradient are refused."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        out = moe.rms_norm(x, w)
        ctx.save_for_backward(x, w, out["rstd"])
        return out["y"]

    @staticmethod
    def backward(ctx, gy):
        x, w, rstd = ctx.saved_tensors
        g = moe.rms_norm_backward(gy.contiguous(), x, w, rstd)
        return g["grad_sum"], g["grad_w"].to(w.dtype)


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.order = order
        return moe.dispatch(x, order)["rows"]

    @staticmethod
    def backward(ctx, g):
        return moe.dispatch_backward(g.contiguous(), ctx.order), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, p, order):
        ctx.order = order
        ctx.save_for_backward(y, p)
        return moe.combine(y, order, p)

    @staticmethod
    def backward(ctx, g):
        y, p = ctx.saved_tensors
        out = moe.combine_backward(g.contiguous(), y, ctx.order, p)
        return out["grad_y"], out["grad_w"], None


def test_gradients_through_functions():
    T, H, k, E = 40, 256, 3, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, H, generator=g, device="cuda", requires_grad=True)
    w = torch.ones(H, device="cuda", requires_grad=True)
    p = torch.rand(T, k, generator=g, device="cuda", requires_grad=True)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    order = moe.sort_pairs(ids, E, align=8)
    go = torch.randn(T, H, generator=g, device="cuda")
    Combine.apply(Dispatch.apply(Norm.apply(x, w), order), p, order).backward(go)
    with torch.no_grad():
        n = moe.rms_norm(x, w)
        rows = moe.dispatch(n["y"], order)["rows"]
        c = moe.combine_backward(go, rows, order, p)
        want = moe.rms_norm_backward(moe.dispatch_backward(c["grad_y"], order), x, w, n["rstd"])
    assert torch.equal(x.grad, want["grad_sum"]) and torch.equal(w.grad, want["grad_w"]) and torch.equal(p.grad, c["grad_w"])
    # a pair's row is its token's norm.  Off by u = 2^-24: a norm 32 u, a dot product of 256 values fewer than 32 u
    s = x.detach().double()
    terms = go.double() * s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6)
    assert ((p.grad.double() - terms.sum(1, keepdim=True)).abs() <= 2.0 ** -24 * 64 * terms.abs().sum(1, keepdim=True)).all()


def test_tensors_that_require_a_gradient():
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda", requires_grad=True)
    with pytest.raises(moe.MoeError):
        moe.rms_norm(x, w)
    with torch.no_grad():
        want = moe.rms_norm(x, w)["y"]
    assert torch.equal(moe.rms_norm(x, w.detach())["y"], want)
