"""rms_norm and its gradients against the formulas in 64 bits.

Tolerances count roundings, u = 2^-24 being half a step of fp32.  A thread adds
at most 32 squares in a row and a block 10 tree levels, so the sum of squares is
off by less than 48 u, rstd by less than 24 u + 4 u, and n = (s * rstd) * weight
by less than 32 u."""
import numpy as np
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
N_REL = 32 * U
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = {moe.QUANT_E4M3_128: 128, moe.QUANT_MXFP8: 32}


def _half(dt):
    return torch.finfo(dt).eps / 2


def _least(dt):
    """Half the smallest step of a 16-bit type (its subnormals)."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def _inputs(T, H, dt, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(dt)
    r = (3 * torch.randn(T, H, generator=g, device="cuda")).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dt)
    return x, r, w


def _e4m3(v):
    """v (float64) on the E4M3 grid, round to nearest even, saturating."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -40))), -6)
    step = 2.0 ** (e - 3)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def _check_quant(n, q, scales, quant, rel):
    """Codes and scales of n (float64, each value off by at most `rel`): a code is the reference's unless n is that
    near to a rounding border; scales agree to `rel` and two roundings."""
    T, H = n.shape
    G = GROUP.get(quant, H)
    q, scales = q.double().cpu().numpy(), scales.double().cpu().numpy()
    for i in range(-(-H // G)):
        v, c = n[:, i * G:(i + 1) * G], q[:, i * G:(i + 1) * G]
        a = np.abs(v).max(1)
        if quant == moe.QUANT_MXFP8:
            near = 1 + 2 * rel
            lo, hi = (np.clip(np.floor(np.log2(np.maximum(a * f, 2.0 ** -140))) - 8, -127, 127) for f in (1 / near, near))
            s = np.log2(scales[:, i])
            assert ((s == lo) | (s == hi))[a > 0].all() and (s[a == 0] == -127).all()
        else:
            want = np.maximum(a, 2.0 ** -100) / 448
            assert (np.abs(scales[:, i] - want) <= (rel + 2 * U) * want).all()
        u = v / scales[:, i:i + 1]
        # the kernel's quotient: n, the scale's and the factor's rounding, the product's
        d = 2 * rel + 4 * U
        lo, hi = _e4m3(u * (1 - d)), _e4m3(u * (1 + d))
        assert ((c == lo) | (c == hi)).all()


# few rows; then rows enough for the kernels' other splits: a warp a row, one, two and four pieces a thread
SHAPES = [(1, 8), (1, 256), (3, 136), (5, 1840), (2, 2056), (4, 4096), (7, 7168), (3, 16384), (300, 520),
          (310, 8), (310, 136), (2050, 264), (310, 520), (2050, 776), (2049, 1000), (333, 1032), (320, 4104), (310, 16384)]
# several rows a block in the backward pass, in each of its splits
LONG = [(8, 1000), (16, 264), (17, 264), (2, 4104), (3, 4104), (5000, 264), (5001, 1000), (2500, 1024), (1300, 2056), (650, 4104), (640, 7176), (620, 16384)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_against_64_bits(T, H, dtype):
    dt = DTYPES[dtype]
    x, r, w = _inputs(T, H, dt, T * 31 + H)
    x[T - 1] = 0
    if T > 2:
        r[T - 1] = 0                                    # an all-zero row
    out = moe.rms_norm(x, w, residual=r, eps=1e-5)
    exact = x.double() + r.double()
    assert ((out["sum"].double() - exact).abs() <= exact.abs() * (_half(dt) + U) + _least(dt)).all()
    s = out["sum"].double()
    rstd = 1 / torch.sqrt((s * s).mean(1) + 1e-5)
    assert ((out["rstd"].double() - rstd).abs() <= 28 * U * rstd).all()
    n = s * rstd[:, None] * w.double()
    assert ((out["y"].double() - n).abs() <= n.abs() * (_half(dt) + N_REL) + _least(dt)).all()
    assert out["y"][T - 1].float().abs().sum() == 0 if T > 2 else True
    # without the residual: the norm of x itself
    alone = moe.rms_norm(out["sum"], w, eps=1e-5)
    assert set(alone) == {"y", "rstd"}
    assert torch.equal(alone["y"], out["y"]) and torch.equal(alone["rstd"], out["rstd"])


@pytest.mark.parametrize("quant", [moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW, moe.QUANT_MXFP8])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_8_bit_output(T, H, dtype, quant):
    dt = DTYPES[dtype]
    x, r, w = _inputs(T, H, dt, T * 17 + H)
    x[:, : H // 4] *= 0.01                              # groups of different size
    if T > 2:
        x[1], r[1] = 0, 0
    out = moe.rms_norm(x, w, residual=r, quant=quant)
    s = out["sum"].double()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * w.double()
    _check_quant(n.cpu().numpy(), out["q"], out["scales"], quant, N_REL)
    # the same values next to an output in the rows' type
    both = dict(y=torch.empty_like(x), q=torch.empty_like(out["q"]), scales=torch.empty_like(out["scales"]))
    moe.rms_norm(out["sum"], w, quant=quant, out=both)
    assert torch.equal(both["q"].view(torch.uint8), out["q"].view(torch.uint8))
    assert torch.equal(both["scales"].view(torch.uint8), out["scales"].view(torch.uint8))
    assert torch.equal(both["y"], moe.rms_norm(out["sum"], w)["y"])


@pytest.mark.parametrize("quant", [moe.QUANT_NONE, moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW, moe.QUANT_MXFP8])
def test_norm_rows_that_are_not_finite_stay_alone(quant):
    x, _, w = _inputs(4, 1024, torch.bfloat16, 5, residual=False)
    good = moe.rms_norm(x, w, quant=quant)
    x[1, 3] = float("nan")
    x[2, 700] = float("inf")
    bad = moe.rms_norm(x, w, quant=quant)
    name = "y" if quant == moe.QUANT_NONE else "q"
    a, b = good[name].float(), bad[name].float()
    assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
    assert b[1].isnan().all()                           # the statistic is NaN
    assert b[2, 700].isnan()                            # inf * 0
    if quant == moe.QUANT_NONE:
        assert (b[2, :700] == 0).all() and (b[2, 701:] == 0).all()
    elif quant == moe.QUANT_MXFP8:
        sc = bad["scales"].view(torch.uint8)
        assert (sc[1] == 255).all() and sc[2, 700 // 32] == 255 and (sc[2, : 700 // 32] == 0).all()
        assert b[2, 700 // 32 * 32: 700 // 32 * 32 + 32].isnan().all()
    else:
        assert bad["scales"][1].isnan().all()


@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-20, 1e-40])
@pytest.mark.parametrize("quant", [moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW, moe.QUANT_MXFP8])
def test_norm_8_bit_output_of_groups_next_to_nothing(quant, eps):
    """Zero rows, zero groups and groups below the scale's bound of 2^-100, whatever rstd is."""
    H = 512
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(5, H, generator=g, device="cuda") * 2.0 ** -40
    x[0] = 0
    x[1, :256] = 0
    x[2, 128:] *= 2.0 ** -60
    x[3] *= 2.0 ** -50
    w = torch.ones(H, device="cuda")
    w[256:384] = 2.0 ** -20
    out = moe.rms_norm(x, w, eps=eps, quant=quant)
    s = x.double()
    # eps as the kernel gets it: rounded to fp32
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(np.float32(eps))) * w.double()
    # squares below 2^-126 lose bits: up to half of 2^-149 each, against a sum of at least H * eps
    rel = N_REL + 2.0 ** -150 / float(np.float32(eps))
    _check_quant(n.cpu().numpy(), out["q"], out["scales"], quant, rel)
    assert (out["q"][0].float() == 0).all() and out["scales"].float().isfinite().all()


def test_norm_of_values_whose_squares_leave_fp32():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = moe.rms_norm(torch.full((1, 64), 1e25, dtype=torch.bfloat16, device="cuda"), w)
    assert out["rstd"].item() == 0 and (out["y"] == 0).all()


@pytest.mark.parametrize("T,H", [(9, 712), (2100, 712), (400, 2064)])
def test_norm_strided_rows_and_in_place(T, H):
    dt = torch.bfloat16
    x, r, w = _inputs(T, H, dt, 3)
    want = moe.rms_norm(x, w, residual=r)
    wide = torch.full((T, 3 * H), float("nan"), dtype=dt, device="cuda")
    wide[:, H:2 * H] = x
    wide2 = torch.full((T, 2 * H), float("nan"), dtype=dt, device="cuda")
    wide2[:, :H] = r
    got = moe.rms_norm(wide[:, H:2 * H], w, residual=wide2[:, :H])
    for name in want:
        assert torch.equal(got[name], want[name]), name
    stream = r.clone()                                   # the residual stream updated where it is
    got = moe.rms_norm(x, w, residual=stream, out=dict(sum=stream, y=torch.empty_like(x)))
    assert torch.equal(stream, want["sum"]) and torch.equal(got["y"], want["y"])
    got = moe.rms_norm(x, w, residual=r, out=dict(y=torch.empty_like(x)))   # the sum is not wanted
    assert torch.equal(got["y"], want["y"])


def test_norm_of_no_rows():
    x = torch.empty(0, 256, dtype=torch.float16, device="cuda")
    w = torch.ones(256, dtype=torch.float16, device="cuda")
    out = moe.rms_norm(x, w, quant=moe.QUANT_MXFP8)
    assert out["q"].shape == (0, 256)
    g = moe.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert g["grad_sum"].shape == (0, 256) and (g["grad_w"] == 0).all()


def _grads(T, H, dt, seed, with_sum):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = (2 * torch.randn(T, H, generator=g, device="cuda")).to(dt)
    gy = torch.randn(T, H, generator=g, device="cuda").to(dt)
    gs = torch.randn(T, H, generator=g, device="cuda").to(dt) if with_sum else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dt)
    return s, gy, gs, w


@pytest.mark.parametrize("with_sum", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,H", SHAPES + [(1000, 256)] + LONG)
def test_norm_backward_against_64_bits(T, H, dtype, with_sum):
    dt = DTYPES[dtype]
    s, gy, gs, w = _grads(T, H, dt, T + H, with_sum)
    rstd = moe.rms_norm(s, w)["rstd"]
    out = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
    r = rstd.double()[:, None]
    n, g = s.double() * r, gy.double() * w.double()
    add = gs.double() if with_sum else torch.zeros_like(n)
    want = r * (g - n * (g * n).mean(1, keepdim=True)) + add
    # g and n: one rounding each; their products' mean 48; the last three operations
    tol = 64 * U * (r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + add.abs())
    assert ((out["grad_sum"].double() - want).abs() <= tol + want.abs() * _half(dt) + _least(dt)).all()
    p = gy.double() * n
    # a column's additions: its rows of one block in a row, the blocks' sums in eight chains
    assert ((out["grad_w"].double() - p.sum(0)).abs() <= (T / 256 + 64) * U * p.abs().sum(0)).all()
    again = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
    assert torch.equal(again["grad_w"], out["grad_w"]) and torch.equal(again["grad_sum"], out["grad_sum"])


def test_norm_backward_against_differences():
    """Central differences of the 64-bit forward, the whole gradient along random directions."""
    T, H, eps, h = 6, 264, 1e-5, 1e-5
    s, gy, gs, w = _grads(T, H, torch.float32, 11, True)
    rstd = moe.rms_norm(s, w, eps=eps)["rstd"]
    out = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)

    def loss(s64, w64):
        n = s64 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + eps)
        return ((gy.double() * n * w64).sum() + (gs.double() * s64).sum()).item()

    g = torch.Generator(device="cuda").manual_seed(12)
    for _ in range(4):
        ds = torch.randn(T, H, generator=g, device="cuda", dtype=torch.float64)
        dw = torch.randn(H, generator=g, device="cuda", dtype=torch.float64)
        num = (loss(s.double() + h * ds, w.double() + h * dw) - loss(s.double() - h * ds, w.double() - h * dw)) / (2 * h)
        terms = torch.cat([(out["grad_sum"].double() * ds).reshape(-1), out["grad_w"].double() * dw])
        # fp32 gradients: 70 u of each term; the difference: h^2 of third derivatives and 2^-52 / h of the loss
        size = abs(loss(s.double(), w.double())) + terms.abs().sum().item()
        assert abs(num - terms.sum().item()) <= 70 * U * 4 * terms.abs().sum().item() + (h * h * 100 + 2.0 ** -50 / h) * size


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm_backward_into_part_of_a_gradient_buffer(dtype):
    """grad_w aligned to its element only, for one row, a few and many."""
    for T, H in ((1, 1032), (4, 4104), (8, 264), (700, 2056)):
        s, gy, gs, w = _grads(T, H, DTYPES[dtype], T, True)
        rstd = moe.rms_norm(s, w)["rstd"]
        want = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
        flat = torch.full((H + 8,), 7.0, device="cuda")
        out = dict(grad_sum=torch.empty_like(s), grad_w=flat[3:3 + H])
        moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs, out=out)
        assert torch.equal(out["grad_w"], want["grad_w"]) and torch.equal(out["grad_sum"], want["grad_sum"])
        assert (flat[:3] == 7).all() and (flat[3 + H:] == 7).all()


def test_norm_backward_in_place():
    for T, H in ((400, 1024), (700, 2048), (1300, 4096)):
        s, gy, gs, w = _grads(T, H, torch.bfloat16, 1, True)
        rstd = moe.rms_norm(s, w)["rstd"]
        want = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
        for at in ("gy", "gs"):
            a, b = gy.clone(), gs.clone()
            out = dict(grad_sum=a if at == "gy" else b, grad_w=torch.empty(H, device="cuda"))
            moe.rms_norm_backward(a, s, w, rstd, grad_sum=b, out=out)
            assert torch.equal(out["grad_sum"], want["grad_sum"]) and torch.equal(out["grad_w"], want["grad_w"])


def test_norm_on_another_stream_and_in_a_graph():
    T, H = 64, 2048
    x, r, w = _inputs(T, H, torch.bfloat16, 21)
    want = moe.rms_norm(x, w, residual=r, quant=moe.QUANT_E4M3_128)
    back = moe.rms_norm_backward(x, want["sum"], w, want["rstd"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.rms_norm(x, w, residual=r, quant=moe.QUANT_E4M3_128, stream=side)
    gback = moe.rms_norm_backward(x, got["sum"], w, got["rstd"], stream=side)
    side.synchronize()
    for name in want:
        assert torch.equal(got[name].view(torch.uint8), want[name].view(torch.uint8)), name
    assert torch.equal(gback["grad_w"], back["grad_w"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.rms_norm(x, w, residual=r, quant=moe.QUANT_E4M3_128)
        gback = moe.rms_norm_backward(x, got["sum"], w, got["rstd"])
    x.copy_(torch.roll(x, 1, 0))
    r.copy_(torch.roll(r, 1, 0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["sum"], torch.roll(want["sum"], 1, 0))
    assert torch.equal(got["q"].view(torch.uint8), torch.roll(want["q"].view(torch.uint8), 1, 0))
    assert torch.equal(gback["grad_sum"], torch.roll(back["grad_sum"], 1, 0))


def test_norm_backward_workspaces_do_not_meet():
    """The call's workspace inside a graph, under eager allocations between replays, and on two streams at once."""
    T, H = 700, 2048
    s, gy, gs, w = _grads(T, H, torch.bfloat16, 41, True)
    rstd = moe.rms_norm(s, w)["rstd"]
    want = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
    again = moe.rms_norm_backward(want["grad_sum"], s, w, rstd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs)
        between = torch.zeros(1 << 22, device="cuda") + 5
        two = moe.rms_norm_backward(one["grad_sum"], s, w, rstd)
    for _ in range(10):
        graph.replay()
        torch.full((1 << 20,), 3.0, device="cuda")
    torch.cuda.synchronize()
    assert (between == 5).all()
    for a, b in ((one, want), (two, again)):
        assert torch.equal(a["grad_w"], b["grad_w"]) and torch.equal(a["grad_sum"], b["grad_sum"])
    side = torch.cuda.Stream()
    got = [moe.rms_norm_backward(gy, s, w, rstd, grad_sum=gs, stream=st) for _ in range(30) for st in (None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a["grad_w"], want["grad_w"]) for a in got)
