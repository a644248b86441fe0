"""One transformer block's mixture-of-experts half around the package's token path.

    python examples/moe_block.py          # needs a GB300; a few seconds

serve():  residual + norm -> route -> sort -> dispatch of 8-bit rows with their scales -> the caller's own
          expert products -> combine with the residual stream; beside it the same block on `Plan.forward`.
train():  the block's forward pass, its gradients through the package's backward entry points, and a few steps of
          gradient descent.

The experts' products are torch matmuls here: they stand for whatever products the caller has.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_routed_expert_router_gb300 as moe  # noqa: E402


class Weights:
    """A block's weights: norm [H], router [E][H] fp32, experts' gate, up [E][I][H] and down [E][H][I]."""

    def __init__(self, H, E, I, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

        bf = torch.bfloat16
        self.norm = normal(H, std=0.1, dtype=torch.float32).add_(1).to(bf)
        self.router = normal(E, H, std=H ** -0.5, dtype=torch.float32)
        self.gate, self.up = normal(E, I, H, std=H ** -0.5, dtype=bf), normal(E, I, H, std=H ** -0.5, dtype=bf)
        self.down = normal(E, H, I, std=I ** -0.5, dtype=bf)


def segments(order):
    """(expert, first row, end) of the experts that have rows."""
    at = order["expert_offsets"].tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(at, at[1:])) if b > a]


def experts(w, rows, order):
    """Every expert's gate, up, SwiGLU and down product of its segment of rows."""
    y, saved = torch.zeros_like(rows), []
    for e, a, b in segments(order):
        x = rows[a:b]
        g, u = x @ w.gate[e].T, x @ w.up[e].T
        h = (torch.nn.functional.silu(g.float()) * u.float()).to(x.dtype)
        y[a:b] = h @ w.down[e].T
        saved.append((e, a, b, g, u, h))
    return y, saved


def experts_backward(w, rows, saved, grad_y):
    """Gradients of rows and of the three stacked weights."""
    grad_rows = torch.zeros_like(rows)
    grads = {n: torch.zeros(getattr(w, n).shape, device="cuda") for n in ("gate", "up", "down")}
    for e, a, b, g, u, h in saved:
        gy, gf, uf = grad_y[a:b], g.float(), u.float()
        gh = (gy @ w.down[e]).float()
        s = torch.sigmoid(gf)
        gu = (gh * gf * s).to(rows.dtype)
        gg = (gh * uf * s * (1 + gf * (1 - s))).to(rows.dtype)
        grads["down"][e] = (gy.T @ h).float()
        grads["gate"][e], grads["up"][e] = (gg.T @ rows[a:b]).float(), (gu.T @ rows[a:b]).float()
        grad_rows[a:b] = gg @ w.gate[e] + gu @ w.up[e]
    return grad_rows, grads


def forward(w, plan, x, stream, E):
    """stream' = stream + x, out = stream' + MoE(norm(stream')); returns what the backward pass needs."""
    n = moe.rms_norm(x, w.norm, residual=stream)
    routed = plan.route(n["y"], w.router)
    order = moe.sort_pairs(routed["topk_ids"], E, align=16)
    rows = moe.dispatch(n["y"], order)["rows"]
    y, saved = experts(w, rows, order)
    out = moe.combine(y, order, routed["topk_w"], base=n["sum"])
    return out, (n, routed, order, rows, y, saved)


def backward(w, grad_out, state):
    """Gradients of x (and of the stream it is added to) and of the block's weights."""
    n, routed, order, rows, y, saved = state
    ids, p = routed["topk_ids"].long(), routed["topk_w"]
    back = moe.combine_backward(grad_out, y, order, p)           # base's gradient is grad_out itself
    grad_rows, grads = experts_backward(w, rows, saved, back["grad_y"])
    grad_y = moe.dispatch_backward(grad_rows, order).float()
    # the router: weights renormalised over the chosen experts
    g = p * (back["grad_w"] - (back["grad_w"] * p).sum(1, keepdim=True))
    T, k = ids.shape
    grads["router"] = torch.zeros_like(w.router).index_add_(
        0, ids.reshape(-1), (g[:, :, None] * n["y"].float()[:, None, :]).reshape(T * k, -1))
    grad_y += (g[:, :, None] * w.router[ids]).sum(1)
    last = moe.rms_norm_backward(grad_y.to(n["y"].dtype), n["sum"], w.norm, n["rstd"], grad_sum=grad_out)
    grads["norm"] = last["grad_w"]
    return last["grad_sum"], grads


def train(T=320, H=512, E=16, I=256, k=4, steps=20, lr=0.05):
    """Gradient descent on a fixed batch; returns the losses and the first step's state, for checks."""
    w = Weights(H, E, I)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, stream = (torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    target = torch.randn(T, H, generator=g, device="cuda")
    losses, first = [], None
    with moe.Plan(H, 128, E, k, T) as plan:
        for _ in range(steps):
            out, state = forward(w, plan, x, stream, E)
            diff = out.float() - target
            losses.append((diff * diff).mean().item())
            grad_out = (diff / H).to(torch.bfloat16)
            grad_x, grads = backward(w, grad_out, state)
            if first is None:
                first = dict(w=Weights(H, E, I), x=x, stream=stream, out=out, grad_out=grad_out, grad_x=grad_x, grads=grads,
                             ids=state[1]["topk_ids"].long())
            for name, grad in grads.items():
                t = getattr(w, name)
                t.copy_((t.float() - lr * grad.float() * H / T).to(t.dtype))
        assert plan.sync_status() == moe.OK
    return losses, first


def serve(T=64, H=512, E=16, I=256, k=4):
    """One prompt through the block twice: expert products of 8-bit rows by the caller, and Plan.forward's FP4 ones.
    Returns both outputs and the same in fp32 from the unquantised weights."""
    w = Weights(H, E, I, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, stream = (torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    with moe.Plan(H, I, E, k, T) as plan:
        n = moe.rms_norm(x, w.norm, residual=stream)
        routed = plan.route(n["y"], w.router)
        order = moe.sort_pairs(routed["topk_ids"], E, align=16)

        q = moe.rms_norm(n["sum"], w.norm, quant=moe.QUANT_E4M3_128)
        d = moe.dispatch(q["q"], order, scales=q["scales"])
        rows = (d["rows"].float() * d["scales"].repeat_interleave(128, 1)).to(torch.bfloat16)   # the products' operand
        own = moe.combine(experts(w, rows, order)[0], order, routed["topk_w"], base=n["sum"])

        fp4 = moe.ExpertSet(*(moe.quantize_nvfp4(t.float().contiguous()) for t in (w.gate, w.up, w.down)))
        planned = plan.forward(n["y"], w.router, None, fp4) + n["sum"]
        assert plan.sync_status() == moe.OK

    y = n["y"].float()
    each = torch.stack([(torch.nn.functional.silu(y @ a.float().T) * (y @ b.float().T)) @ c.float().T
                        for a, b, c in zip(w.gate, w.up, w.down)], 1)                  # [T][E][H]
    picked = torch.gather(each, 1, routed["topk_ids"].long()[:, :, None].expand(-1, -1, H))
    exact = (picked * routed["topk_w"][:, :, None]).sum(1) + n["sum"].float()
    return own, planned, exact


def off(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


if __name__ == "__main__":
    own, planned, exact = serve()
    print(f"serve: 8-bit rows, own products {off(own, exact):.4f} off fp32; Plan.forward (NVFP4 weights) {off(planned, exact):.4f}")
    losses, _ = train()
    print("train: loss " + " ".join(f"{v:.3f}" for v in losses))
