"""head_norm and its gradients where a row holds an infinity, at every place of a row: what the formulas give in 64 bits.
A value that is not rotated has no partner, so nothing of it reaches another value but through the row's mean."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_head_norm import DTYPES, EPS, inputs, normed, reference_gradients, rotate

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (128, 64), (80, 16), (48, 32), (112, 96), (64, 0), (96, 96), (512, 256)]
INF = float("inf")


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D,R", SHAPES)
def test_an_infinity_anywhere_in_a_row(D, R, dtype, pairs):
    """Token t's infinity is at place t.  The norm of every finite value is 0, the infinity's own a NaN."""
    q, k, qw, kw, pos = inputs(D, 3, 1, D, DTYPES[dtype], D + R)
    t = torch.arange(D, device="cuda")
    q[t, 1, t] = INF
    k[t, 0, t] = -INF
    out = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(R), interleaved=pairs, eps=EPS)
    for name, x, w in (("q", q, qw), ("k", k, kw)):
        want = rotate(normed(x)[0] * w.double(), pos, R, pairs)[0]
        assert torch.equal(out[name].isnan(), want.isnan())
        assert (out[name][want == 0] == 0).all()
    assert out["q"][:, 1][~out["q"][:, 1].isnan()].abs().sum() == 0
    clean = moe.head_norm(torch.where(q.isinf(), 0, q), k, qw, kw, pos, moe.rotary_turns(R), interleaved=pairs, eps=EPS)
    assert torch.equal(out["q"][:, ::2], clean["q"][:, ::2])


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("what", ["grad", "weight", "x"])
def test_an_infinity_in_a_backward_pass(D, R, dtype, pairs, what):
    """One at a time, at the last places and in the middle of the part that does not turn (of the rotated part where all do)."""
    turns = moe.rotary_turns(R)
    for d in {D - 1, (D + R) // 2 if R < D else D // 2, R if R < D else 0}:
        q, k, qw, kw, pos = inputs(40, 3, 2, D, DTYPES[dtype], D + R)
        gq, gk, *_ = inputs(40, 3, 2, D, DTYPES[dtype], D + R + 1)
        if what == "grad":
            gq[7, 1, d] = INF
        elif what == "x":
            q[7, 1, d] = INF
        else:
            qw[d] = INF
        out = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns, interleaved=pairs, eps=EPS)
        gx, tol, gw, total = reference_gradients(gq, q, qw, pos, R, pairs)
        got = out["grad_qw"].double()
        fine = gw.isfinite()
        assert fine.sum() >= D - 2 and torch.equal(got.isfinite(), fine)
        assert ((got - gw).abs() <= 512 * 2.0 ** -24 * total)[fine].all()            # test_gpu_head_norm's depth for 120 rows is below 320
        assert torch.equal(out["grad_q"].isfinite(), gx.isfinite())
        there = gx.isfinite()
        half = torch.finfo(q.dtype).eps / 2
        assert ((out["grad_q"].double() - gx).abs() <= gx.abs() * half + tol + torch.finfo(q.dtype).smallest_normal * half)[there].all()
        assert out["grad_k"].isfinite().all() and out["grad_kw"].isfinite().all()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,R", SHAPES)
def test_an_infinite_weight(D, R, pairs):
    q, k, qw, kw, pos = inputs(5, 2, 1, D, torch.float32, D + R)
    qw[D - 1] = INF
    out = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(R), interleaved=pairs, eps=EPS)["q"]
    want = rotate(normed(q)[0] * qw.double(), pos, R, pairs)[0]
    assert torch.equal(out.isfinite(), want.isfinite())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,R", SHAPES)
def test_an_infinite_weight_in_a_row_with_an_infinity(D, R, pairs):
    """0 times the infinite weight is a NaN there as well."""
    q, k, qw, kw, pos = inputs(D, 2, 1, D, torch.float32, D + R)
    t = torch.arange(D, device="cuda")
    q[t, 1, t] = INF
    qw[D - 1], qw[D // 2] = INF, float("nan")
    out = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(R), interleaved=pairs, eps=EPS)["q"]
    want = rotate(normed(q)[0] * qw.double(), pos, R, pairs)[0]
    assert torch.equal(out[:, 1].isnan(), want[:, 1].isnan())
