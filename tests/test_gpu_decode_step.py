"""The decode step of examples/decode_block.py: each call's result against its formula in 64 bits on the inputs that it
had in the run, the whole step in a replayed graph, and the head norm under autograd."""
import os
import sys
from types import SimpleNamespace

import pytest
import torch

import moe_routed_expert_router_gb300 as moe
import test_gpu_decode_layer as layer_test
import test_gpu_head_norm as head_test
import test_gpu_linear as linear_test

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block as example  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def tokens(seed, S=4, H=1024):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(S, H, generator=g, device="cuda").to(BF), torch.randn(S, H, generator=g, device="cuda").to(BF)


def without_ts(w):
    return moe.NvfpTensor(w.codes, w.scales, w.ts)


def test_every_call_of_a_step():
    b = example.Block()
    for at in range(3):
        x, stream = tokens(at)
        out, s = example.decode(b, x, stream, at)
        nq, nk = b.heads, b.kv_heads
        linear_test.check(s["raw"].view(4, -1), s["n1"]["y"], without_ts(b.qkv))
        for name, w, rows in (("q", b.q_norm, s["raw"][:, :nq]), ("k", b.k_norm, s["raw"][:, nq:nq + nk])):
            n = head_test.normed(rows)[0]                       # with this file's eps below, head_norm's own is 1e-6
            x64 = rows.double()
            n = x64 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + 1e-6) * w.double()
            y, size = head_test.rotate(n, s["position"], b.D, False, base=1e6)
            assert ((s[name].double() - y).abs() <= y.abs() * 2 ** -8 + 32 * head_test.U * size * 1.01).all()
        assert torch.equal(b.keys[:, at], s["k"]) and torch.equal(b.values[:, at], s["raw"][:, nq + nk:])
        assert (b.keys[:, at + 1:] == 0).all()                  # nothing written behind the new row
        linear_test.check(s["y"], s["attention"], without_ts(b.proj))
        L = SimpleNamespace(x=s["n2"]["y"], rw=b.router, bias=None, gate=b.experts[0], up=b.experts[1], down=b.experts[2], shared=b.shared,
                            base=s["n2"]["sum"], k=b.k, dt=BF, router=moe.ROUTER_SOFTMAX, renorm=True)
        layer_test.check(L, s["layer"])
        assert torch.equal(out, s["layer"]["out"])


def test_a_step_replayed():
    b = example.Block(seed=3)
    x, stream = tokens(5)
    example.decode(b, x, stream, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = example.decode(b, x, stream, 1)
    for seed in (6, 7):
        x2, stream2 = tokens(seed)
        x.copy_(x2)
        stream.copy_(stream2)
        graph.replay()
        torch.cuda.synchronize()
        got, keys = out.clone(), b.keys[:, 1].clone()
        want, _ = example.decode(b, x, stream, 1)
        assert torch.equal(got, want) and torch.equal(keys, b.keys[:, 1])


def test_head_norm_under_autograd():
    """Gradients through the Function are the entry point's, with shared weights added and expanded gradients taken."""
    T, nq, nk, D = 40, 4, 2, 64
    q, k, w, _, pos = head_test.inputs(T, nq, nk, D, torch.float32, 8)
    turns = moe.rotary_turns(D)
    gq, gk, *_ = head_test.inputs(T, nq, nk, D, torch.float32, 9)
    want = moe.head_norm_backward(gq, gk, q, k, w, w, pos, turns)
    q.requires_grad_(), k.requires_grad_(), w.requires_grad_()
    with pytest.raises(moe.MoeError):
        moe.head_norm(q, k, w, w, pos, turns)
    a, b = example.HeadNorm.apply(q, k, w, w, pos, turns)
    torch.autograd.backward((a, b), (gq, gk))
    assert torch.equal(q.grad, want["grad_q"]) and torch.equal(k.grad, want["grad_k"])
    assert torch.equal(w.grad, want["grad_qw"] + want["grad_kw"])
    q.grad = k.grad = w.grad = None
    a, b = example.HeadNorm.apply(q, k, w, w, pos, turns)
    (a.sum() + 2 * b.sum()).backward()                            # gradients of stride zero
    again = moe.head_norm_backward(torch.ones_like(gq), torch.full_like(gk, 2.0), q.detach(), k.detach(), w.detach(), w.detach(), pos, turns)
    assert torch.equal(q.grad, again["grad_q"]) and torch.equal(k.grad, again["grad_k"])


def test_the_example_runs():
    import subprocess
    r = subprocess.run([sys.executable, example.__file__], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
