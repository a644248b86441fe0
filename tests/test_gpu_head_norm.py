"""head_norm and its gradients against the formulas in 64 bits.

Tolerances count roundings, u = 2^-24 being half a step of fp32.  A lane adds 16 squares and the row's lanes five tree
levels, so the mean square is off by less than 23 u, rstd by less than 13 u and n = x * w * rstd by less than 16 u.  An
angle is rounded once, in half turns: up to 2^-25 of one, 1.6 u radians; the sine and cosine are off by two steps at most,
4 u; the two products and the sum of a plane add 3 u.  So a rotated value is off by less than (16 + 1.6 + 4 + 3) u of
|a| + |b|: 32 u is allowed.  The frequencies' own rounding (2^-52 of the angle) stays below 2^-30 for positions to 2^21."""
import math

import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def half(dt):
    return torch.finfo(dt).eps / 2


def least(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def inputs(T, Hq, Hk, D, dt, seed=0, far=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dt)
    pos = torch.randint(-5, 1 << (21 if far else 10), (T,), generator=g, device="cuda", dtype=torch.int32)
    return normal(T, Hq, D, std=2), normal(T, Hk, D), (1 + normal(D, std=0.3).float()).to(dt), (1 + normal(D, std=0.3).float()).to(dt), pos


def frequencies(R, base=1e4):
    return [base ** (-2.0 * i / R) for i in range(R // 2)]


def planes(x, R, pairs):
    """The rotated values as [..][R/2][2]."""
    return x[..., :R].unflatten(-1, (R // 2, 2)) if pairs else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)


def unplanes(z, rest, pairs):
    return torch.cat([(z if pairs else z.transpose(-1, -2)).flatten(-2), rest], -1)


def rotate(x, pos, R, pairs, sign=1.0, base=1e4):
    """Rotation in 64 bits, and |a| + |b| of every value's plane (the value's own size where it is not rotated)."""
    if R == 0:
        return x, x.abs()
    a = pos.double()[:, None, None] * torch.tensor(frequencies(R, base), dtype=torch.float64, device=x.device)
    z = planes(x, R, pairs)
    c, s = torch.cos(a), sign * torch.sin(a)
    y = torch.stack([z[..., 0] * c - z[..., 1] * s, z[..., 1] * c + z[..., 0] * s], -1)
    size = z.abs().sum(-1, keepdim=True).expand_as(z)
    return unplanes(y, x[..., R:], pairs), unplanes(size, x[..., R:].abs(), pairs)


def normed(x):
    x = x.double()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def check(got, x, w, pos, R, pairs):
    n = normed(x)[0] * w.double()
    y, size = rotate(n, pos, R, pairs)
    assert ((got.double() - y).abs() <= y.abs() * half(got.dtype) + 32 * U * size * (1 + half(got.dtype)) + least(got.dtype)).all()


# tokens, query and key heads, D, R: every count of lanes a row, idle lanes, no and partial rotation, tiles of one and
# several tokens, a last tile that is not full, many and few heads
SHAPES = [(1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (5, 3, 2, 48, 32), (4, 40, 1, 64, 64), (37, 7, 5, 80, 80),
          (311, 24, 24, 96, 64), (700, 1, 1, 256, 16), (129, 12, 4, 192, 0), (64, 2, 1, 512, 512), (3001, 5, 1, 112, 96),
          (2, 1024, 3, 16, 16), (1500, 9, 16, 128, 128)]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
def test_against_64_bits(T, Hq, Hk, D, R, dtype, pairs):
    dt = DTYPES[dtype]
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, dt, T + D)
    q[T - 1, Hq - 1] = 0                                          # an all-zero row
    out = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(R), interleaved=pairs, eps=EPS)
    check(out["q"], q, qw, pos, R, pairs)
    check(out["k"], k, kw, pos, R, pairs)
    assert out["q"][T - 1, Hq - 1].float().abs().sum() == 0


def test_far_positions_turn_exactly():
    """Positions whose angle an fp32 product would miss by whole radians."""
    D, base = 64, 1e6
    pos = torch.tensor([0, 1, 1 << 20, (1 << 21) - 1, -1, -(1 << 20)], dtype=torch.int32, device="cuda")
    q, k, qw, kw, _ = inputs(len(pos), 2, 2, D, torch.float32, 3)
    out = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(D, base), eps=EPS)
    y, size = rotate(normed(q)[0] * qw.double(), pos, D, False, base=base)
    assert ((out["q"].double() - y).abs() <= 32 * U * size + U * y.abs()).all()
    # frequencies of the caller's own
    scaled = [f / 8 for f in frequencies(D, base)]
    same = moe.head_norm(q, k, qw, kw, pos, moe.rotary_turns(D, frequencies=scaled), eps=EPS)
    slow = moe.head_norm(q, k, qw, kw, pos // 8, moe.rotary_turns(D, base), eps=EPS)
    at = (pos % 8 == 0).nonzero()[:, 0]
    assert (same["q"][at] - slow["q"][at]).abs().max() <= 64 * U * size.max()


def test_the_largest_positions_wrap_whole_turns():
    """At position 2^31 - 1 the product is taken in integers: checked against the same in Python's."""
    D, R = 16, 16
    for p in (2 ** 31 - 1, -2 ** 31):
        q = torch.zeros(1, 1, D, device="cuda")
        q[0, 0, 0:8] = 1.0                                       # a = 1, b = 0 in every plane
        one = torch.ones(D, device="cuda")
        turns = moe.rotary_turns(R)
        y = moe.head_norm(q, q, one, one, torch.tensor([p], dtype=torch.int32, device="cuda"), turns, eps=1e-12)["q"][0, 0]
        for i, t in enumerate(turns.tolist()):
            turn = (p * t) % 2 ** 64 / 2 ** 64
            size = 2 ** 0.5                                      # 1 / sqrt(mean square), the mean being 1 / 2
            assert abs(y[i].item() - size * math.cos(2 * math.pi * turn)) <= 32 * U * size
            assert abs(y[i + 8].item() - size * math.sin(2 * math.pi * turn)) <= 32 * U * size


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_parts_of_one_products_rows(dtype):
    """Strided inputs and outputs, in place, and nothing written beside them."""
    dt, T, Hq, Hk, D = DTYPES[dtype], 33, 6, 2, 96
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    _, _, qw, kw, pos = inputs(T, 1, 1, D, dt, 2)
    turns = moe.rotary_turns(64)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    want = moe.head_norm(q.contiguous(), k.contiguous(), qw, kw, pos, turns)
    got = moe.head_norm(q, k, qw, kw, pos, turns)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])
    cache = torch.full((T, 3, Hk, D), 7.0, dtype=dt, device="cuda")
    moe.head_norm(q, k, qw, kw, pos, turns, out=dict(q=torch.empty_like(want["q"]), k=cache[:, 1]))
    assert torch.equal(cache[:, 1], want["k"]) and (cache[:, 0] == 7).all() and (cache[:, 2] == 7).all()
    values = qkv[:, Hq + Hk:].clone()
    moe.head_norm(q, k, qw, kw, pos, turns, out=dict(q=q, k=k))   # in place
    assert torch.equal(q, want["q"]) and torch.equal(k, want["k"]) and torch.equal(qkv[:, Hq + Hk:], values)


def test_rows_that_are_not_finite_stay_alone():
    q, k, qw, kw, pos = inputs(4, 8, 2, 64, torch.bfloat16, 5)
    turns = moe.rotary_turns(64)
    good = moe.head_norm(q, k, qw, kw, pos, turns)
    q[1, 3, 5], q[2, 0, 0] = float("nan"), float("inf")
    bad = moe.head_norm(q, k, qw, kw, pos, turns)
    assert bad["q"][1, 3].isnan().all() and bad["q"][2, 0, 0].isnan() and torch.equal(bad["k"], good["k"])
    rest = torch.ones(4, 8, dtype=torch.bool, device="cuda")
    rest[1, 3] = rest[2, 0] = False
    assert torch.equal(bad["q"][rest], good["q"][rest])


def reference_gradients(gy, x, w, pos, R, pairs):
    """Gradients in 64 bits; with what their tolerances are counted in."""
    n, rstd = normed(x)
    g, size = rotate(gy.double(), pos, R, pairs, sign=-1.0)
    gw, sw = g * w.double(), size * w.double().abs()
    mean = (gw * n).mean(-1, keepdim=True)
    gx = rstd * (gw - n * mean)
    # g is off by 9 u of |a| + |b|, the mean by (9 + 25 + 13) u of the sum of magnitudes, the rest by 20 u
    tol = 80 * U * rstd * (sw + n.abs() * (sw * n.abs()).mean(-1, keepdim=True))
    return gx, tol, (g * n).sum((0, 1)), (size * n.abs()).sum((0, 1))


def check_gradients(out, gq, gk, q, k, qw, kw, pos, R, pairs):
    for name, gy, x, w in (("q", gq, q, qw), ("k", gk, k, kw)):
        gx, tol, gw, total = reference_gradients(gy, x, w, pos, R, pairs)
        got = out["grad_" + name]
        assert ((got.double() - gx).abs() <= gx.abs() * half(got.dtype) + tol + least(got.dtype)).all(), name
        # terms off by 9 + 13 u and a product's rounding; a chain of adds: a thread's rows, up to 256 groups of a block,
        # 8 of up to 512 blocks and two levels of 8
        rows = x.shape[0] * x.shape[1]
        depth = 32 + rows // 256 + 256 + 8 + 16
        assert ((out[f"grad_{name}w"].double() - gw).abs() <= depth * U * total).all(), name


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
def test_gradients_against_64_bits(T, Hq, Hk, D, R, dtype, pairs):
    dt = DTYPES[dtype]
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, dt, T + D)
    gq, gk, *_ = inputs(T, Hq, Hk, D, dt, T + D + 1)
    turns = moe.rotary_turns(R)
    out = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns, interleaved=pairs, eps=EPS)
    check_gradients(out, gq, gk, q, k, qw, kw, pos, R, pairs)
    again = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns, interleaved=pairs, eps=EPS)
    for name in out:
        assert torch.equal(out[name], again[name])               # a fixed order of sums


def test_gradients_against_differences():
    """The slope of sum(gy * y) along a direction, by differences of the definition in 64 bits."""
    T, Hq, Hk, D, R = 6, 3, 2, 64, 48
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, torch.float32, 11)
    gq, gk, *_ = inputs(T, Hq, Hk, D, torch.float32, 12)
    out = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, moe.rotary_turns(R), eps=EPS)
    g = torch.Generator(device="cuda").manual_seed(13)
    for name, gy, x, w in (("q", gq, q, qw), ("k", gk, k, kw)):
        def loss(x, w):
            return (rotate(normed(x)[0] * w, pos, R, False)[0] * gy.double()).sum()
        dx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        dw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        h, x64, w64 = 1e-5, x.double(), w.double()
        tol = reference_gradients(gy, x, w, pos, R, False)[1]
        slope = (loss(x64 + h * dx, w64) - loss(x64 - h * dx, w64)) / (2 * h)
        # the third derivative times h^2 / 6, and 64-bit cancellation over h: both far below 1e-6
        assert abs((out["grad_" + name].double() * dx).sum() - slope) <= (tol * dx.abs()).sum() + 1e-6
        slope = (loss(x64, w64 + h * dw) - loss(x64, w64 - h * dw)) / (2 * h)
        total = reference_gradients(gy, x, w, pos, R, False)[3]
        assert abs((out[f"grad_{name}w"].double() * dw).sum() - slope) <= (400 * U * total * dw.abs()).sum() + 1e-6


def test_gradients_in_place_and_strided():
    T, Hq, Hk, D = 50, 4, 2, 128
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, torch.bfloat16, 21)
    gq, gk, *_ = inputs(T, Hq, Hk, D, torch.bfloat16, 22)
    turns = moe.rotary_turns(D)
    want = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns)
    wide = torch.cat([q, k, k], 1)
    got = moe.head_norm_backward(gq, gk, wide[:, :Hq], wide[:, Hq:Hq + Hk], qw, kw, pos, turns)
    for name in want:
        assert torch.equal(got[name], want[name])
    own = dict(want, grad_q=gq, grad_k=k, grad_qw=torch.empty(D, device="cuda"), grad_kw=torch.empty(D, device="cuda"))
    moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns, out=own)      # over a gradient and over an input
    for name in want:
        assert torch.equal(own[name], want[name])


def test_no_tokens():
    q, k, qw, kw, pos = inputs(2, 2, 1, 32, torch.float32)
    turns = moe.rotary_turns(32)
    out = moe.head_norm(q[:0], k[:0], qw, kw, pos[:0], turns)
    assert out["q"].shape == (0, 2, 32)
    back = moe.head_norm_backward(q[:0], k[:0], q[:0], k[:0], qw, kw, pos[:0], turns,
                                  out=dict(grad_q=q[:0], grad_k=k[:0], grad_qw=torch.ones(32, device="cuda"), grad_kw=torch.ones(32, device="cuda")))
    assert (back["grad_qw"] == 0).all() and (back["grad_kw"] == 0).all()


def test_rows_past_four_gigabytes():
    """Offsets in bytes beyond 32 bits: a token stride of 64 MB in a buffer of 70 tokens."""
    T, Hq, Hk, D, stride = 70, 2, 1, 64, 1 << 25
    store = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, torch.bfloat16, 31)
    rows = store.view(T, stride)
    far_q, far_k = rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, 4096:4096 + Hk * D].unflatten(1, (Hk, D))
    far_q.copy_(q)
    far_k.copy_(k)
    turns = moe.rotary_turns(D)
    want = moe.head_norm(q, k, qw, kw, pos, turns)
    got = moe.head_norm(far_q, far_k, qw, kw, pos, turns)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])


def test_captured_and_replayed_on_another_stream():
    T, Hq, Hk, D = 400, 8, 2, 128
    q, k, qw, kw, pos = inputs(T, Hq, Hk, D, torch.bfloat16, 41)
    gq, gk, *_ = inputs(T, Hq, Hk, D, torch.bfloat16, 42)
    turns = moe.rotary_turns(D)
    moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.head_norm(q, k, qw, kw, pos, turns)
        back = moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns)
    for seed in (43, 44):
        q2, k2, *_ = inputs(T, Hq, Hk, D, torch.bfloat16, seed)
        q.copy_(q2)
        k.copy_(k2)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        want, wback = moe.head_norm(q, k, qw, kw, pos, turns, stream=side), moe.head_norm_backward(gq, gk, q, k, qw, kw, pos, turns, stream=side)
        side.synchronize()
        for a, b in ((out, want), (back, wback)):
            for name in a:
                assert torch.equal(a[name], b[name])


def test_workspaces_of_calls_behind_one_another():
    """Gradients of different sizes, nothing waiting between them: each has the memory of the one before."""
    cases = []
    for T, Hq, Hk, D in ((900, 8, 2, 64), (37, 3, 1, 128), (2500, 4, 4, 32), (300, 16, 2, 256)):
        q, k, qw, kw, pos = inputs(T, Hq, Hk, D, torch.bfloat16, T)
        gq, gk, *_ = inputs(T, Hq, Hk, D, torch.bfloat16, T + 1)
        cases.append((gq, gk, q, k, qw, kw, pos, moe.rotary_turns(D)))
    want = [{n: t.clone() for n, t in moe.head_norm_backward(*c).items()} for c in cases]
    got = [moe.head_norm_backward(*c) for _ in range(5) for c in cases]
    for i, out in enumerate(got):
        for name in out:
            assert torch.equal(out[name], want[i % 4][name])
