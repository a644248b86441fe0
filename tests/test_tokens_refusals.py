"""What the norm, sort, dispatch and combine entry points refuse, before anything is launched (no GPU needed)."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

A, NULL = 256, None      # an aligned address that is never used, and none
INV, SHAPE, ALIGN = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED_SHAPE, moe.ERR_MISALIGNED


def norm(x=A, xs=256, r=NULL, rs=0, w=A, T=4, H=256, dt=moe.DTYPE_BF16, eps=1e-6, quant=moe.QUANT_NONE, s=NULL, y=A,
         q=NULL, sc=NULL, rstd=NULL):
    return moe.lib().moe_rms_norm(x, xs, r, rs, w, T, H, dt, eps, quant, s, y, q, sc, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=3), INV), (dict(dt=-1), INV), (dict(H=0), SHAPE), (dict(H=252), SHAPE),
    (dict(H=16392, xs=16392), SHAPE), (dict(xs=248), SHAPE), (dict(xs=260), SHAPE), (dict(r=A, rs=128), SHAPE),
    (dict(quant=4), INV), (dict(quant=-1), INV), (dict(eps=0.0), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(x=NULL), INV), (dict(w=NULL), INV),
    (dict(y=NULL), INV), (dict(s=A), INV), (dict(q=A), INV), (dict(sc=A), INV),
    (dict(quant=moe.QUANT_MXFP8, q=A), INV), (dict(quant=moe.QUANT_E4M3_128, sc=A), INV),
    (dict(x=A + 8), ALIGN), (dict(w=A + 2), ALIGN), (dict(y=A + 8), ALIGN), (dict(r=A + 8, rs=256), ALIGN),
    (dict(rstd=A + 2), ALIGN), (dict(quant=moe.QUANT_E4M3_ROW, q=A + 8, sc=A), ALIGN),
    (dict(quant=moe.QUANT_E4M3_ROW, q=A, sc=A + 1), ALIGN), (dict(T=0), moe.OK)])
def test_norm(kw, want):
    assert norm(**kw) == want


def norm_back(gy=A, s=A, w=A, rstd=A, gs=NULL, T=400, H=256, dt=moe.DTYPE_BF16, gi=A, gw=A, ws=A, n=1 << 30):
    return moe.lib().moe_rms_norm_backward(gy, s, w, rstd, gs, T, H, dt, gi, gw, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=9), INV), (dict(H=20), SHAPE), (dict(gy=NULL), INV), (dict(s=NULL), INV),
    (dict(w=NULL), INV), (dict(rstd=NULL), INV), (dict(gi=NULL), INV), (dict(gw=NULL), INV), (dict(ws=NULL), INV),
    (dict(n=0), INV), (dict(gs=A + 8), ALIGN), (dict(gi=A + 8), ALIGN), (dict(ws=A + 8), ALIGN),
    (dict(rstd=A + 1), ALIGN), (dict(gw=A + 1), ALIGN)])
def test_norm_backward(kw, want):
    assert norm_back(**kw) == want


def test_norm_backward_workspace():
    n = moe.lib().moe_rms_norm_backward_workspace
    assert n(0, 256) == 0 and n(-1, 256) == 0
    assert n(400, 256) > 0 and norm_back(n=n(400, 256) - 1) == INV
    assert n(1, 256) == 0 and n(1, 4096) == 0           # one block's sums are the result
    assert n(1 << 20, 16384) == n(1 << 30, 16384)


def test_sorted_rows():
    n = moe.lib().moe_sorted_rows
    assert n(0, 8, 128) == 0 and n(32, 128, 1) == 32
    assert n(32, 128, 128) == 32 * 128              # every pair may have an expert of its own
    assert n(1000, 4, 16) == (1000 + 4 * 15) // 16 * 16
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, 0), (8, 8, 3), (8, 8, 512), (1 << 31, 8, 1)):
        assert n(*bad) == -1
    with pytest.raises(moe.MoeError) as e:
        moe.sorted_rows(8, 8, 3)
    assert e.value.status == SHAPE


def sort(ids=A, T=4, k=8, E=16, align=1, rows=32, off=A, sr=A, pr=A):
    return moe.lib().moe_sort_pairs(ids, T, k, E, align, rows, off, sr, pr, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(align=3), SHAPE), (dict(align=512), SHAPE), (dict(rows=31), INV), (dict(rows=33), INV), (dict(rows=-1), INV),
    (dict(T=1 << 30, k=4), SHAPE), (dict(T=(1 << 31) - 1, k=1, rows=(1 << 31) + 15, align=2), SHAPE),
    (dict(ids=NULL), INV), (dict(off=NULL), INV), (dict(sr=NULL), INV), (dict(pr=NULL), INV), (dict(ids=A + 2), ALIGN),
    (dict(off=A + 1), ALIGN), (dict(sr=A + 2), ALIGN), (dict(pr=A + 3), ALIGN)])
def test_sort_pairs(kw, want):
    assert sort(**kw) == want


def dispatch(x=A, xs=512, rb=512, sc=NULL, sb=0, T=4, k=8, sr=A, pr=A, rows=32, out=A, osc=NULL):
    return moe.lib().moe_dispatch(x, xs, rb, sc, sb, T, k, sr, pr, rows, out, osc, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(rows=-1), INV), (dict(k=0), SHAPE), (dict(rb=0), SHAPE), (dict(rb=520, xs=528), SHAPE),
    (dict(xs=496), SHAPE), (dict(xs=520), SHAPE), (dict(rb=1 << 40, xs=1 << 40), SHAPE), (dict(sc=A, sb=4), INV),
    (dict(osc=A, sb=4), INV), (dict(sc=A, osc=A), INV), (dict(sb=4), INV), (dict(sb=-4), SHAPE), (dict(x=NULL), INV),
    (dict(sr=NULL), INV), (dict(pr=NULL), INV), (dict(out=NULL), INV), (dict(x=A + 8), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(sr=A + 2), ALIGN), (dict(pr=A + 2), ALIGN), (dict(rows=0, T=0), moe.OK)])
def test_dispatch(kw, want):
    assert dispatch(**kw) == want


def combine(y=A, dt=moe.DTYPE_BF16, T=4, k=8, H=256, pr=A, rows=32, w=A, base=NULL, out=A):
    return moe.lib().moe_combine(y, dt, T, k, H, pr, rows, w, base, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=5), INV), (dict(k=33), SHAPE), (dict(H=12), SHAPE), (dict(H=0), SHAPE),
    (dict(rows=-1), INV), (dict(rows=1 << 31), SHAPE), (dict(y=NULL), INV), (dict(pr=NULL), INV), (dict(out=NULL), INV),
    (dict(y=A + 8), ALIGN), (dict(base=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(pr=A + 2), ALIGN),
    (dict(w=A + 2), ALIGN), (dict(T=0), moe.OK)])
def test_combine(kw, want):
    assert combine(**kw) == want


def combine_back(go=A, y=A, dt=moe.DTYPE_BF16, T=4, k=8, H=256, sr=A, pr=A, rows=32, w=A, gy=A, gw=A):
    return moe.lib().moe_combine_backward(go, y, dt, T, k, H, sr, pr, rows, w, gy, gw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(dt=5), INV), (dict(k=0), SHAPE), (dict(H=12), SHAPE), (dict(go=NULL), INV),
    (dict(y=NULL), INV), (dict(sr=NULL), INV), (dict(pr=NULL), INV), (dict(w=NULL), INV), (dict(gy=NULL), INV),
    (dict(gw=NULL), INV), (dict(go=A + 8), ALIGN), (dict(y=A + 8), ALIGN), (dict(gy=A + 8), ALIGN),
    (dict(sr=A + 2), ALIGN), (dict(pr=A + 2), ALIGN), (dict(w=A + 2), ALIGN), (dict(gw=A + 2), ALIGN),
    (dict(T=0), moe.OK)])
def test_combine_backward(kw, want):
    assert combine_back(**kw) == want


def test_binding_refuses_tensors_the_kernels_cannot_take():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    order = dict(sorted_rows=torch.zeros(8, dtype=torch.int32), pair_rows=ids)
    for call in (lambda: moe.rms_norm(x, w), lambda: moe.rms_norm(x.double(), w), lambda: moe.rms_norm(x[0], w),
                 lambda: moe.rms_norm_backward(x, x, w, w[:4]), lambda: moe.sort_pairs(ids, 4),
                 lambda: moe.sort_pairs(ids.reshape(-1), 4), lambda: moe.dispatch(x, order),
                 lambda: moe.combine(x, order), lambda: moe.combine_backward(x, x, order, x[:, :2])):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == INV
