"""What head_norm, linear_fp4 and decode_layer refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import moe_routed_expert_router_gb300 as moe

A, NULL = 256, None      # an aligned address that is never used, and none
INV, SHAPE, ALIGN = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED_SHAPE, moe.ERR_MISALIGNED


def head(q=A, qs=512, k=A, ks=128, qw=A, kw=A, pos=A, turns=A, T=4, Hq=8, Hk=2, D=64, R=64, il=0, dt=moe.DTYPE_BF16, eps=1e-6, qo=A,
         qos=512, ko=A, kos=128):
    return moe.lib().moe_head_norm(q, qs, k, ks, qw, kw, pos, turns, T, Hq, Hk, D, R, il, dt, eps, qo, qos, ko, kos, None)


HEADS = [
    (dict(T=-1), INV), (dict(dt=3), INV), (dict(il=2), INV), (dict(il=-1), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(Hq=0), SHAPE), (dict(Hk=0), SHAPE), (dict(Hq=1025, qs=65600), SHAPE), (dict(D=0), SHAPE),
    (dict(D=56), SHAPE), (dict(D=528, R=64, qs=5000, ks=5000), SHAPE), (dict(R=-16), SHAPE), (dict(R=80), SHAPE), (dict(R=24), SHAPE),
    (dict(qs=504), SHAPE), (dict(qs=516), SHAPE), (dict(ks=120), SHAPE), (dict(q=NULL), INV), (dict(k=NULL), INV), (dict(qw=NULL), INV),
    (dict(kw=NULL), INV), (dict(pos=NULL), INV), (dict(turns=NULL), INV), (dict(q=A + 8), ALIGN), (dict(k=A + 8), ALIGN),
    (dict(qw=A + 2), ALIGN), (dict(kw=A + 4), ALIGN), (dict(pos=A + 2), ALIGN), (dict(turns=A + 4), ALIGN)]


@pytest.mark.parametrize("kw,want", HEADS + [
    (dict(qos=504), SHAPE), (dict(kos=132), SHAPE), (dict(qo=NULL), INV), (dict(ko=NULL), INV), (dict(qo=A + 8), ALIGN),
    (dict(ko=A + 8), ALIGN), (dict(T=0), moe.OK)])
def test_head_norm(kw, want):
    assert head(**kw) == want


def head_back(gq=A, gqs=512, gk=A, gks=128, q=A, qs=512, k=A, ks=128, qw=A, kw=A, pos=A, turns=A, T=4, Hq=8, Hk=2, D=64, R=64, il=0,
              dt=moe.DTYPE_BF16, eps=1e-6, oq=A, ok=A, oqw=A, okw=A, ws=A, n=1 << 30):
    return moe.lib().moe_head_norm_backward(gq, gqs, gk, gks, q, qs, k, ks, qw, kw, pos, turns, T, Hq, Hk, D, R, il, dt, eps, oq, ok,
                                            oqw, okw, ws, n, None)


@pytest.mark.parametrize("kw,want", HEADS + [
    (dict(gqs=504), SHAPE), (dict(gks=130), SHAPE), (dict(gq=NULL), INV), (dict(gk=NULL), INV), (dict(oq=NULL), INV), (dict(ok=NULL), INV),
    (dict(oqw=NULL), INV), (dict(okw=NULL), INV), (dict(T=4000, ws=NULL), INV), (dict(T=4000, n=0), INV), (dict(gq=A + 8), ALIGN),
    (dict(gk=A + 8), ALIGN), (dict(oq=A + 8), ALIGN), (dict(ok=A + 8), ALIGN), (dict(oqw=A + 2), ALIGN), (dict(okw=A + 1), ALIGN),
    (dict(ws=A + 8), ALIGN), (dict(T=0, oqw=NULL), INV)])
def test_head_norm_backward(kw, want):
    assert head_back(**kw) == want


def test_head_norm_backward_workspace():
    n = moe.lib().moe_head_norm_backward_workspace
    assert n(0, 8, 2, 64, 64) == 0 and n(-1, 8, 2, 64, 64) == 0 and n(4, 8, 2, 60, 32) == 0
    assert n(1, 1, 1, 64, 64) == 0                                # one block of each: their sums are the result
    assert n(4000, 8, 2, 64, 64) > 0 and head_back(T=4000, n=n(4000, 8, 2, 64, 64) - 1) == INV
    assert n(1 << 20, 8, 2, 64, 64) == n(1 << 30, 8, 2, 64, 64)


def weight(codes=A, scales=A, ts=A):
    return moe.Nvfp4(codes, scales, ts)


def linear(x=A, xs=256, w=weight(), fmt=moe.WEIGHTS_NVFP4, T=4, N=64, K=256, dt=moe.DTYPE_BF16, to=moe.DTYPE_BF16, out=A, ws=NULL,
           n=0):
    return moe.lib().moe_linear_fp4(x, xs, None if w is None else ctypes.byref(w), fmt, T, N, K, dt, to, out, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=moe.DTYPE_F32, to=moe.DTYPE_F32), INV), (dict(dt=7), INV), (dict(to=moe.DTYPE_F16), INV), (dict(to=5), INV),
    (dict(fmt=2), INV), (dict(fmt=-1), INV), (dict(w=None), INV), (dict(N=0), SHAPE), (dict(N=(1 << 31) - 1), SHAPE), (dict(K=0), SHAPE),
    (dict(K=192), SHAPE), (dict(K=65664, xs=65664), SHAPE), (dict(xs=248), SHAPE), (dict(xs=260), SHAPE), (dict(T=(1 << 20) + 1), SHAPE),
    (dict(x=NULL), INV), (dict(out=NULL), INV), (dict(w=weight(codes=NULL)), INV), (dict(w=weight(scales=NULL)), INV),
    (dict(w=weight(ts=NULL)), INV), (dict(x=A + 8), ALIGN), (dict(w=weight(codes=A + 8)), ALIGN), (dict(w=weight(scales=A + 4)), ALIGN),
    (dict(w=weight(ts=A + 2)), ALIGN), (dict(out=A + 1), ALIGN), (dict(to=moe.DTYPE_F32, out=A + 2), ALIGN), (dict(T=0), moe.OK)])
def test_linear(kw, want):
    assert linear(**kw) == want


def test_linear_workspace():
    """Large products want one and refuse to run without it."""
    n = moe.lib().moe_linear_fp4_workspace
    nv, mx = moe.WEIGHTS_NVFP4, moe.WEIGHTS_MXFP4
    assert n(nv, 0, 1 << 17, 256) == 0 and n(nv, 16, 0, 256) == 0 and n(nv, (1 << 20) + 1, 1 << 17, 256) == 0
    assert n(nv, 16, 1 << 17, 384) == 0 and n(mx, 16, 1 << 17, 256) == 0      # rows of scales of whole 16 bytes
    assert n(nv, 16, (1 << 17) - 1, 256) == 0 and n(nv, 8, 1 << 17, 256) == 0
    big = dict(T=16, N=1 << 17, K=256)
    want = n(nv, 16, 1 << 17, 256)
    assert want >= 16 * 8 * 256 // 2
    assert linear(**big) == INV and linear(**big, ws=A, n=want - 1) == INV and linear(**big, n=want) == INV
    assert linear(**big, ws=A + 128, n=want) == ALIGN
    for T in (17, 255, 256, 257, 300, 1 << 20):                   # more tokens go in pieces of 256
        assert n(nv, T, 1 << 16, 1024) <= n(nv, 256, 1 << 16, 1024) + n(nv, T % 256 or 256, 1 << 16, 1024)


def layer(x=A, dt=moe.DTYPE_BF16, T=4, H=256, rw=A, rdt=0, bias=NULL, E=16, k=4, router=0, renorm=1, gate=A, up=A, down=A, I=64, sg=NULL,
          su=NULL, sd=NULL, Is=0, base=NULL, out=A, ids=A, w=A, ws=A, n=1 << 30):
    return moe.lib().moe_decode_layer(x, dt, T, H, rw, rdt, bias, E, k, router, renorm, gate, up, down, I, sg, su, sd, Is, base, out, ids,
                                      w, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=3), INV), (dict(rdt=2), INV), (dict(router=2), INV), (dict(renorm=2), INV), (dict(T=17), SHAPE),
    (dict(H=0), SHAPE), (dict(H=252), SHAPE), (dict(H=16392), SHAPE), (dict(I=0), SHAPE), (dict(I=60), SHAPE), (dict(I=16392), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33, E=64), SHAPE), (dict(k=17), SHAPE), (dict(Is=-8), SHAPE),
    (dict(Is=12, sg=A, su=A, sd=A), SHAPE), (dict(x=NULL), INV), (dict(rw=NULL), INV), (dict(gate=NULL), INV), (dict(up=NULL), INV),
    (dict(down=NULL), INV), (dict(out=NULL), INV), (dict(ids=NULL), INV), (dict(w=NULL), INV), (dict(ws=NULL), INV), (dict(n=0), INV),
    (dict(sg=A), INV), (dict(Is=64, sg=A, su=A), INV), (dict(x=A + 8), ALIGN), (dict(rw=A + 4), ALIGN), (dict(gate=A + 8), ALIGN),
    (dict(down=A + 2), ALIGN), (dict(ws=A + 8), ALIGN), (dict(base=A + 1), ALIGN), (dict(out=A + 1), ALIGN), (dict(bias=A + 2), ALIGN),
    (dict(ids=A + 2), ALIGN), (dict(w=A + 2), ALIGN), (dict(dt=moe.DTYPE_F32, out=A + 2), ALIGN), (dict(T=0), moe.OK)])
def test_layer(kw, want):
    assert layer(**kw) == want


def test_layer_workspace():
    n = moe.lib().moe_decode_layer_workspace
    assert n(0, 16, 64, 4, 0) == 0 and n(17, 16, 64, 4, 0) == 0 and n(4, 16, 64, 33, 0) == 0
    assert n(4, 16, 64, 4, 64) >= 4 * (4 * 16 + 4 * 4 * 64 + 4 * 64)
    assert layer(n=n(4, 16, 64, 4, 0) - 1) == INV


@pytest.mark.parametrize("call", [
    lambda: moe.rotary_turns(24), lambda: moe.rotary_turns(-16), lambda: moe.rotary_turns(32, frequencies=[1.0] * 15),
    lambda: moe.rotary_turns(32, frequencies=[float("nan")] * 16), lambda: moe.rotary_turns(32, base=0.0), lambda: moe.rotary_turns(32, base=-5.0),
    lambda: moe.rotary_turns(32, base=float("inf"))])
def test_rotary_turns_refuses(call):
    with pytest.raises(moe.MoeError):
        call()


def test_rotary_turns():
    t = moe.rotary_turns(32, base=10000.0, device="cpu")
    assert t.dtype is torch.int64 and t.shape == (16,)
    for i, v in enumerate(t.tolist()):
        assert abs((v % 2 ** 64) / 2 ** 64 * 2 * 3.141592653589793 - 10000.0 ** (-2 * i / 32)) < 1e-15
    whole = moe.rotary_turns(16, frequencies=[2 * 3.141592653589793 * (3 + 0.25)] * 8, device="cpu")       # whole turns drop out
    assert all(abs(v / 2 ** 64 - 0.25) < 1e-15 for v in whole.tolist())
    assert moe.rotary_turns(0, device="cpu").shape == (0,)


def test_binding_refuses_tensors_the_kernels_cannot_take():
    x, pos, turns, w = torch.zeros(4, 2, 32), torch.zeros(4, dtype=torch.int32), torch.zeros(16, dtype=torch.int64), torch.zeros(32)
    t = moe.NvfpTensor(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 8, dtype=torch.uint8), torch.zeros(1))
    rows, e = torch.zeros(4, 128), torch.zeros(2, 8, 128)
    for call in (lambda: moe.head_norm(x, x, w, w, pos, turns), lambda: moe.head_norm(x[0], x, w, w, pos, turns),
                 lambda: moe.head_norm_backward(x, x, x, x, w, w, pos, turns), lambda: moe.linear_fp4(rows.half(), t),
                 lambda: moe.linear_fp4(rows[0], t), lambda: moe.decode_layer(rows, rows[:2], e, e, e.mT, 1),
                 lambda: moe.decode_layer(rows[0], rows[:2], e, e, e.mT, 1)):
        with pytest.raises(moe.MoeError) as err:
            call()
        assert err.value.status == INV
