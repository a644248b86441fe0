"""One transformer block's decode step on the package's calls, and the training pass of its head norm.

    python examples/decode_block.py       # needs a GB300; a few seconds

decode(): residual + norm -> queries, keys and values by one 4-bit product -> head norm with the rotation, in place, the
          new keys straight into the cache -> the caller's attention -> the 4-bit product back -> residual + norm -> the
          whole mixture-of-experts layer with its shared expert, added to the stream.
HeadNorm: head_norm for autograd, through head_norm_backward.

The attention is plain torch here: it stands for whatever attention the caller has.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_routed_expert_router_gb300 as moe  # noqa: E402

BF = torch.bfloat16


class Block:
    """A block's weights, a cache of keys and values [S][L][heads][D] for S sequences, and the rotation."""

    def __init__(self, S=4, L=64, H=1024, heads=8, kv_heads=2, D=128, E=16, I=256, k=4, shared=256, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype=BF):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
        self.heads, self.kv_heads, self.D, self.k = heads, kv_heads, D, k
        self.norm1, self.norm2 = (normal(H, std=0.1, dtype=torch.float32).add_(1).to(BF) for _ in range(2))
        self.q_norm, self.k_norm = (normal(D, std=0.1, dtype=torch.float32).add_(1).to(BF) for _ in range(2))
        self.qkv = moe.quantize_nvfp4(normal((heads + 2 * kv_heads) * D, H, std=H ** -0.5, dtype=torch.float32))
        self.proj = moe.quantize_mxfp4(normal(H, heads * D, std=(heads * D) ** -0.5, dtype=torch.float32))
        self.router = normal(E, H, std=H ** -0.5, dtype=torch.float32)
        self.experts = (normal(E, I, H, std=H ** -0.5), normal(E, I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5))
        self.shared = (normal(shared, H, std=H ** -0.5), normal(shared, H, std=H ** -0.5), normal(H, shared, std=shared ** -0.5))
        self.turns = moe.rotary_turns(D, base=1e6)
        self.keys, self.values = (torch.zeros(S, L, kv_heads, D, dtype=BF, device="cuda") for _ in range(2))


def attention(q, keys, values, length):
    """q [S][heads][D] over the first `length` cached rows."""
    S, heads, D = q.shape
    n = heads // keys.shape[2]
    k = keys[:, :length].float().repeat_interleave(n, 2)
    v = values[:, :length].float().repeat_interleave(n, 2)
    p = torch.softmax(torch.einsum("shd,slhd->shl", q.float(), k) * D ** -0.5, -1)
    return torch.einsum("shl,slhd->shd", p, v).to(BF).reshape(S, heads * D)


def decode(b, x, stream, at):
    """One new token of every sequence, x and stream [S][H], at position `at` of all: the stream behind the block, and what the steps
    between gave, by name."""
    S, nq, nk, D = x.shape[0], b.heads, b.kv_heads, b.D
    n1 = moe.rms_norm(x, b.norm1, residual=stream)
    qkv = moe.linear_fp4(n1["y"], b.qkv).view(S, nq + 2 * nk, D)
    position = torch.full((S,), at, dtype=torch.int32, device="cuda")
    raw = qkv.clone()
    new = moe.head_norm(qkv[:, :nq], qkv[:, nq:nq + nk], b.q_norm, b.k_norm, position, b.turns,
                        out=dict(q=qkv[:, :nq], k=b.keys[:, at]))
    b.values[:, at] = qkv[:, nq + nk:]
    a = attention(new["q"], b.keys, b.values, at + 1)
    y = moe.linear_fp4(a, b.proj)
    n2 = moe.rms_norm(y, b.norm2, residual=n1["sum"])
    m = moe.decode_layer(n2["y"], b.router, *b.experts, b.k, shared=b.shared, base=n2["sum"])
    return m["out"], dict(n1=n1, raw=raw, q=new["q"], k=b.keys[:, at], position=position, attention=a, y=y, n2=n2, layer=m)


class HeadNorm(torch.autograd.Function):
    """head_norm of q and k as autograd follows it."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, turns):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, turns)
        out = moe.head_norm(q, k, q_weight, k_weight, positions, turns)
        return out["q"], out["k"]

    @staticmethod
    def backward(ctx, grad_q, grad_k):
        q, k, qw, kw, positions, turns = ctx.saved_tensors
        g = moe.head_norm_backward(grad_q.contiguous(), grad_k.contiguous(), q, k, qw, kw, positions, turns)
        return g["grad_q"], g["grad_k"], g["grad_qw"].to(qw.dtype), g["grad_kw"].to(kw.dtype), None, None


if __name__ == "__main__":
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    stream = torch.randn(4, 1024, generator=g, device="cuda").to(BF)
    for step in range(8):
        x = torch.randn(4, 1024, generator=g, device="cuda").to(BF)
        stream, _ = decode(block, x, stream, step)
    print("decode: 8 steps of 4 sequences, stream's root mean square %.3f" % stream.float().square().mean().sqrt())
    q = torch.randn(32, 8, 128, generator=g, device="cuda", requires_grad=True)
    k = torch.randn(32, 2, 128, generator=g, device="cuda", requires_grad=True)
    w = torch.ones(128, device="cuda", requires_grad=True)
    a, b = HeadNorm.apply(q, k, w, w, torch.arange(32, dtype=torch.int32, device="cuda"), block.turns)
    (a.square().sum() + b.sum()).backward()
    print("train: gradients of queries %.3f, keys %.3f, weight %.3f" % (q.grad.norm(), k.grad.norm(), w.grad.norm()))
