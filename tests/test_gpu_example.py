"""The example block: its gradients against autograd in 64 bits, its 8-bit path against fp32, and that it learns."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu


def test_block_gradients_against_autograd():
    losses, f = moe_block.train(steps=2)
    w = {n: getattr(f["w"], n).double().requires_grad_() for n in ("norm", "router", "gate", "up", "down")}
    x = f["x"].double().requires_grad_()
    s = x + f["stream"].double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * w["norm"]
    logits = torch.gather(y @ w["router"].T, 1, f["ids"])
    p = torch.softmax(logits, 1)
    each = torch.einsum("tei,ehi->teh", torch.nn.functional.silu(torch.einsum("th,eih->tei", y, w["gate"]))
                        * torch.einsum("th,eih->tei", y, w["up"]), w["down"])
    picked = torch.gather(each, 1, f["ids"][:, :, None].expand(-1, -1, x.shape[1]))
    out = s + (picked * p[:, :, None]).sum(1)
    out.backward(f["grad_out"].double())
    # bf16 all along: about ten roundings of half a step (2^-8) on the way to a gradient, of values that
    # are independent, so their relative size stays below ten of them added up
    limit = 10 * 2.0 ** -8
    assert moe_block.off(f["out"], out.detach()) < limit
    assert moe_block.off(f["grad_x"], x.grad) < limit
    for name in w:
        assert moe_block.off(f["grads"][name], w[name].grad) < limit, name


def test_block_learns():
    losses, _ = moe_block.train(steps=20)
    assert losses[-1] < 0.9 * losses[0]
    assert all(b < a for a, b in zip(losses, losses[1:]))


def test_block_serves_8_bit_rows():
    own, planned, exact = moe_block.serve()
    # E4M3: 2^-4 of a value at most, a third of it on average, on the products' input alone
    assert moe_block.off(own, exact) < 2.0 ** -4
    # NVFP4 weights: a value is off by up to a sixth of its block's largest
    assert moe_block.off(planned, exact) < 1 / 6
