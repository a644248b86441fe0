"""sort_pairs, dispatch, combine and their gradients against plain definitions.

Sorting and copies are compared bit for bit; sums against 64 bits, with u = 2^-24
(half a step of fp32) for each of the k + 1 additions and products."""
import numpy as np
import pytest
import torch

import synth
import moe_routed_expert_router_gb300 as moe
from helpers import plan_for

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _half(dt):
    return torch.finfo(dt).eps / 2


def _least(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def _sorted(ids, E, align):
    """The definition, pair by pair."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    P = flat.size
    R = (P + min(E, P) * (align - 1)) // align * align
    kept = (flat >= 0) & (flat < E)
    count = np.bincount(flat[kept], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(-(-count // align) * align)])
    rows, inv = np.full(R, -1, np.int64), np.full(P, -1, np.int64)
    nxt = offsets[:-1].copy()
    for p in np.flatnonzero(kept):
        rows[nxt[flat[p]]] = p
        inv[p] = nxt[flat[p]]
        nxt[flat[p]] += 1
    return offsets, rows, inv.reshape(T, k)


def _ids(T, k, E, seed, drop=0.0, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full((T, k), E - 1)
    elif kind == "none":
        ids = np.full((T, k), -1)
    else:
        p = 1 / np.arange(1, E + 1)
        score = np.log(rng.permutation(p)) + rng.gumbel(size=(T, E))
        ids = np.argsort(-score, axis=1)[:, :k]
    if drop:
        gone = rng.random((T, k)) < drop
        gone[T // 2] = True
        ids = np.where(gone, rng.choice([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31], size=(T, k)), ids)
    return ids.astype(np.int32)


def _check_sort(ids, E, align):
    offsets, rows, inv = _sorted(ids, E, align)
    out = dict(expert_offsets=torch.full((E + 1,), 77, dtype=torch.int32, device="cuda"),
               sorted_rows=torch.full((rows.size,), 77, dtype=torch.int32, device="cuda"),
               pair_rows=torch.full(ids.shape, 77, dtype=torch.int32, device="cuda"))
    moe.sort_pairs(torch.from_numpy(ids).cuda(), E, align=align, out=out)
    np.testing.assert_array_equal(out["expert_offsets"].cpu().numpy(), offsets)
    np.testing.assert_array_equal(out["pair_rows"].cpu().numpy(), inv)
    np.testing.assert_array_equal(out["sorted_rows"].cpu().numpy(), rows)


@pytest.mark.parametrize("align", [1, 8, 128])
@pytest.mark.parametrize("T,k,E,drop,kind", [
    (1, 1, 1, 0, "zipf"), (1, 8, 128, 0, "zipf"), (4, 8, 128, 0, "zipf"), (5, 3, 7, 0.4, "zipf"),
    (33, 1, 2, 0, "zipf"), (129, 10, 500, 0.1, "zipf"), (257, 8, 256, 0, "zipf"), (64, 32, 64, 0, "zipf"),
    (1000, 8, 1024, 0.05, "zipf"), (4093, 7, 255, 0.05, "zipf"), (16384, 8, 256, 0, "zipf"), (20001, 7, 64, 0.05, "zipf"),
    (300, 2, 5, 0, "one"), (4096, 8, 33, 0, "one"), (50, 4, 16, 0, "none"), (5000, 3, 16, 0, "none")])
def test_sort_is_exact(T, k, E, drop, kind, align):
    _check_sort(_ids(T, k, E, T + E, drop, kind), E, align)


@pytest.mark.parametrize("P", [1, 31, 32, 33, 1023, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 8191, 8193, 16385, 16384 * 2 + 1,
                               65536 + 31])
def test_sort_at_the_borders_of_its_split(P):
    rng = np.random.default_rng(P)
    _check_sort(rng.integers(-1, 40, (P, 1)).astype(np.int32), 40, 16)


def test_sort_of_no_tokens():
    out = moe.sort_pairs(torch.empty(0, 8, dtype=torch.int32, device="cuda"), 64, align=128)
    assert out["sorted_rows"].shape == (0,) and out["pair_rows"].shape == (0, 8)
    assert (out["expert_offsets"] == 0).all()


@pytest.mark.parametrize("name", ["decode4_w4a16", "prompt512_w4a16"])
def test_sort_agrees_with_the_router(name):
    w = synth.WORKLOADS[name]
    with plan_for(w) as plan:
        got = plan.route(synth.activations(w, 0, device="cuda"), synth.router_weight(w, 0, "cuda"),
                         synth.router_bias(w, 0, "cuda"))
        assert plan.sync_status() == moe.OK
    order = moe.sort_pairs(got["topk_ids"], w.experts)
    assert torch.equal(order["expert_offsets"], got["expert_offsets"])
    assert torch.equal(order["sorted_rows"], got["sorted_rows"])


CASES = [(1, 1, 4, 1, 0.0), (4, 8, 128, 1, 0.0), (37, 3, 9, 16, 0.3), (130, 10, 40, 128, 0.0), (515, 11, 17, 8, 0.2),
         (90, 32, 64, 1, 0.5)]
# tokens enough for the splits by pairs: two, four, five and eight at a time, and what is left of them
MANY = [(400, k, 24, 8, drop) for k, drop in ((1, 0.0), (2, 0.1), (3, 0.0), (4, 0.3), (5, 0.1), (7, 0.0), (9, 0.1), (10, 0.0),
                                               (16, 0.1), (20, 0.0))]


def _order(T, k, E, align, drop, seed=0):
    return moe.sort_pairs(torch.from_numpy(_ids(T, k, E, seed + T, drop)).cuda(), E, align=align)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "e4m3"])
@pytest.mark.parametrize("H", [16, 144, 1840, 4096])
@pytest.mark.parametrize("T,k,E,align,drop", CASES)
def test_dispatch_copies_rows(T, k, E, align, drop, H, dtype):
    order = _order(T, k, E, align, drop)
    x = torch.randint(0, 256, (T, H * {"e4m3": 1, "f32": 4}.get(dtype, 2)), dtype=torch.uint8, device="cuda")
    x = x.view(DTYPES.get(dtype, torch.float8_e4m3fn))
    scales = {"bf16": None, "f16": torch.randint(0, 256, (T, 7), dtype=torch.uint8, device="cuda"),
              "f32": torch.rand(T, 1, device="cuda"), "e4m3": torch.rand(T, H // 16, device="cuda")}[dtype]
    got = moe.dispatch(x, order, scales=scales)
    rows = order["sorted_rows"].long()

    def want(a):
        b = a.contiguous().view(torch.uint8)
        return torch.where((rows < 0)[:, None], 0, b[rows.clamp(min=0) // k])

    assert torch.equal(got["rows"].view(torch.uint8), want(x))
    if scales is not None:
        assert torch.equal(got["scales"].view(torch.uint8), want(scales))


def test_dispatch_of_strided_rows():
    order = _order(21, 4, 8, 8, 0.2)
    wide = torch.randn(21, 96, device="cuda").to(torch.bfloat16)
    got = moe.dispatch(wide[:, 32:64], order)
    want = moe.dispatch(wide[:, 32:64].contiguous(), order)
    assert torch.equal(got["rows"], want["rows"])


def _pairs64(a, inv):
    """Rows of the pairs in float64, zeros for dropped ones: [T][k][H]."""
    v = a[inv.long().clamp(min=0)].double()
    return torch.where((inv < 0)[:, :, None], 0.0, v)


def _rows_in(order, H, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = torch.randn(order["sorted_rows"].shape[0], H, generator=g, device="cuda").to(dt)
    y[order["sorted_rows"] < 0] = float("nan")           # what no pair holds is not read
    return y


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [8, 136, 1840, 4096])
@pytest.mark.parametrize("T,k,E,align,drop", CASES + MANY)
def test_combine_against_64_bits(T, k, E, align, drop, H, dtype):
    dt = DTYPES[dtype]
    order = _order(T, k, E, align, drop)
    y = _rows_in(order, H, dt, H)
    w = torch.rand(T, k, device="cuda")
    base = torch.randn(T, H, device="cuda").to(dt)
    v = _pairs64(y, order["pair_rows"])
    for weights, add in ((w, None), (w, base), (None, None), (None, base)):
        t = v if weights is None else v * w.double()[:, :, None]
        b = torch.zeros(T, H, dtype=torch.float64, device="cuda") if add is None else add.double()
        want, size = t.sum(1) + b, t.abs().sum(1) + b.abs()
        if weights is None and add is None:
            got = moe.dispatch_backward(y, order)
        else:
            got = moe.combine(y, order, weights, base=add)
        assert ((got.double() - want).abs() <= (k + 1) * U * size + want.abs() * _half(dt) + _least(dt)).all()
    if drop:
        assert (moe.combine(y, order, w)[T // 2] == 0).all()                    # a token without pairs
        assert torch.equal(moe.combine(y, order, w, base=base)[T // 2], base[T // 2])
    stream = base.clone()
    assert torch.equal(moe.combine(y, order, w, base=stream, out=stream), moe.combine(y, order, w, base=base))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [8, 136, 1840, 4096])
@pytest.mark.parametrize("T,k,E,align,drop", CASES + MANY)
def test_combine_backward_against_64_bits(T, k, E, align, drop, H, dtype):
    dt = DTYPES[dtype]
    order = _order(T, k, E, align, drop)
    y = _rows_in(order, H, dt, H + 1)
    w = torch.rand(T, k, device="cuda")
    go = torch.randn(T, H, device="cuda").to(dt)
    got = moe.combine_backward(go, y, order, w)
    rows = order["sorted_rows"].long()
    p = rows.clamp(min=0)
    gy = torch.where((rows < 0)[:, None], 0.0, go.double()[p // k] * w.reshape(-1).double()[p][:, None])
    assert ((got["grad_y"].double() - gy).abs() <= gy.abs() * (_half(dt) + U) + _least(dt)).all()
    terms = _pairs64(y, order["pair_rows"]) * go.double()[:, None, :]
    # a thread's chain of ceil(H / 2048) * 8 products, then 13 tree levels and sums over warps
    tol = (8 * -(-H // 2048) + 24) * U * terms.abs().sum(2)
    assert ((got["grad_w"].double() - terms.sum(2)).abs() <= tol).all()
    assert (got["grad_w"][order["pair_rows"] < 0] == 0).all()
    out = dict(grad_y=y, grad_w=torch.empty(T, k, device="cuda"))             # over y itself
    moe.combine_backward(go, y, order, w, out=out)
    assert torch.equal(y, got["grad_y"]) and torch.equal(out["grad_w"], got["grad_w"])


def test_gradients_against_differences():
    """combine and dispatch are linear in each argument: a difference of two forward results is the gradient's
    product with the step, up to the forward's own roundings."""
    T, k, E, H = 23, 5, 11, 72
    order = _order(T, k, E, 8, 0.2)
    y, w = _rows_in(order, H, torch.float32, 2), torch.rand(T, k, device="cuda")
    go = torch.randn(T, H, device="cuda")
    grads = moe.combine_backward(go, y, order, w)
    dy, dw = _rows_in(order, H, torch.float32, 3), torch.randn(T, k, device="cuda")

    def loss(a, b):
        out = moe.combine(a, order, b)
        return (out.double() * go.double()).sum().item(), (k + 2) * U * (out.abs() * go.abs()).sum().item()

    base, e0 = loss(y, w)
    held = order["sorted_rows"] >= 0
    l1, e1 = loss(y + dy, w)
    size = (k + 4) * U * ((y.abs() + dy.abs())[held].double().sum().item() * go.abs().max().item())
    assert abs(l1 - base - (grads["grad_y"].double() * dy.double())[held].sum().item()) <= e0 + e1 + size
    l2, e2 = loss(y, w + dw)
    kept = order["pair_rows"] >= 0
    size = 64 * U * (w.abs() + dw.abs())[kept].sum().item() * (y[held].abs().sum(1).max() * go.abs().max()).item()
    assert abs(l2 - base - (grads["grad_w"] * dw)[kept].double().sum().item()) <= e0 + e2 + size
    x = torch.randn(T, H, device="cuda")
    rows = moe.dispatch(x, order)["rows"]
    g = torch.where(held[:, None], dy, 0.0)
    back = moe.dispatch_backward(dy, order)
    a, b = (rows.double() * g.double()).sum().item(), (x.double() * back.double()).sum().item()
    assert abs(a - b) <= (k + 1) * U * (rows.abs().double() * g.abs().double()).sum().item()


def test_values_that_are_not_finite_reach_their_token_only():
    order = _order(40, 4, 8, 16, 0.0)
    y = _rows_in(order, 64, torch.bfloat16, 4)
    w = torch.rand(40, 4, device="cuda")
    want = moe.combine(y, order, w)
    row = order["pair_rows"][7, 2].item()
    y[row] = float("inf")
    got = moe.combine(y, order, w)
    assert torch.equal(got[:7], want[:7]) and torch.equal(got[8:], want[8:])
    assert got[7].isinf().all()


def test_entries_out_of_range_count_as_no_pair():
    order = _order(6, 2, 4, 1, 0.0)
    y = torch.randn(12, 32, device="cuda")
    bad = dict(order, pair_rows=order["pair_rows"].clone(), sorted_rows=order["sorted_rows"].clone())
    bad["pair_rows"][3] = torch.tensor([12, -9], dtype=torch.int32)
    bad["pair_rows"][bad["pair_rows"] == 5] = 12      # in both arrays: no pair at row 5
    bad["sorted_rows"][5] = 12
    assert (moe.combine(y, bad)[3] == 0).all()
    assert (moe.dispatch(torch.randn(6, 32, device="cuda"), bad)["rows"][5] == 0).all()
    g = moe.combine_backward(torch.randn(6, 32, device="cuda"), y, bad, torch.rand(6, 2, device="cuda"))
    assert (g["grad_w"][3] == 0).all()


def test_rows_past_4_gb():
    T, k, E, H = 36000, 8, 64, 8192                      # 288000 rows of 16 KB
    g = torch.Generator(device="cuda").manual_seed(9)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    order = moe.sort_pairs(ids, E)
    x = torch.randint(-99, 100, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    rows = moe.dispatch(x, order)["rows"]
    p = order["sorted_rows"].long()
    for a in range(0, T * k, 40000):
        assert torch.equal(rows[a:a + 40000], x[p[a:a + 40000] // k])
    assert torch.equal(moe.dispatch_backward(rows, order).float(), (x.float() * k).to(torch.bfloat16).float())
    w = torch.ones(T, k, device="cuda")
    got = moe.combine_backward(x, rows, order, w, out=dict(grad_y=rows, grad_w=w))
    for a in range(0, T * k, 40000):
        assert torch.equal(got["grad_y"][a:a + 40000], x[p[a:a + 40000] // k])
    exact = x.double().square().sum(1)
    assert ((got["grad_w"].double() - exact[:, None]).abs() <= 56 * U * exact[:, None]).all()


def test_no_tokens():
    order = moe.sort_pairs(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4, align=8)
    x = torch.empty(0, 64, device="cuda")
    assert moe.dispatch(x, order)["rows"].shape == (0, 64)
    assert moe.combine(x, order).shape == (0, 64)
    g = moe.combine_backward(x, x, order, torch.empty(0, 2, device="cuda"))
    assert g["grad_y"].shape == (0, 64) and g["grad_w"].shape == (0, 2)


def test_on_another_stream_and_in_a_graph():
    T, k, E, H = 200, 4, 16, 512
    ids = torch.from_numpy(_ids(T, k, E, 1)).cuda()
    ids2 = torch.from_numpy(_ids(T, k, E, 2, 0.2)).cuda()
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, k, device="cuda")

    def all_of_it(i, stream=None):
        order = moe.sort_pairs(i, E, align=16, stream=stream)
        rows = moe.dispatch(x, order, stream=stream)["rows"]
        out = moe.combine(rows, order, w, base=x, stream=stream)
        g = moe.combine_backward(x, rows, order, w, stream=stream)
        return [order["sorted_rows"], rows, out, g["grad_y"], g["grad_w"],
                moe.dispatch_backward(g["grad_y"], order, stream=stream)]

    want, want2 = all_of_it(ids), all_of_it(ids2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = all_of_it(ids, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = ids.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of_it(static)
    for i, ref in ((ids, want), (ids2, want2), (ids, want)):
        static.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("T,H", [(6, 512), (700, 2048)])
def test_calls_back_to_back(T, H):
    """Launches overlap (each starts while the one before ends): a chain of calls that nothing waits between, over
    changing inputs and the same buffers, gives what the calls give one by one."""
    k, E = 4, 16
    g = torch.Generator(device="cuda").manual_seed(T)
    xs = [torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    ids = [torch.from_numpy(_ids(T, k, E, s, 0.1)).cuda() for s in range(3)]
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    p = torch.rand(T, k, generator=g, device="cuda")
    R = moe.sorted_rows(T * k, E, 8)

    def buffers():
        i32, bf = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        return dict(norm=dict(sum=torch.empty(T, H, **bf), y=torch.empty(T, H, **bf), rstd=torch.empty(T, device="cuda")),
                    order=dict(expert_offsets=torch.empty(E + 1, **i32), sorted_rows=torch.empty(R, **i32),
                               pair_rows=torch.empty(T, k, **i32)),
                    rows=dict(rows=torch.empty(R, H, **bf)), out=torch.empty(T, H, **bf),
                    back=dict(grad_y=torch.empty(R, H, **bf), grad_w=torch.empty(T, k, device="cuda")),
                    gx=torch.empty(T, H, **bf), last=dict(grad_sum=torch.empty(T, H, **bf), grad_w=torch.empty(H, device="cuda")))

    def chain(i, b, wait):
        def step(v):
            if wait:
                torch.cuda.synchronize()
            return v
        n = step(moe.rms_norm(xs[i], w, residual=xs[(i + 1) % 3], out=b["norm"]))
        o = step(moe.sort_pairs(ids[i], E, align=8, out=b["order"]))
        r = step(moe.dispatch(n["y"], o, out=b["rows"]))
        c = step(moe.combine(r["rows"], o, p, base=n["sum"], out=b["out"]))
        back = step(moe.combine_backward(c, r["rows"], o, p, out=b["back"]))
        gx = step(moe.dispatch_backward(back["grad_y"], o, out=b["gx"]))
        last = step(moe.rms_norm_backward(gx, n["sum"], w, n["rstd"], grad_sum=c, out=b["last"]))
        return [c, back["grad_w"], gx, last["grad_sum"], last["grad_w"]]

    want = [[t.clone() for t in chain(i, buffers(), True)] for i in range(3)]
    b, got = buffers(), []
    for n in range(60):
        got.append([t.clone() for t in chain(n % 3, b, False)])
    torch.cuda.synchronize()
    for n, ts in enumerate(got):
        assert all(torch.equal(a, c) for a, c in zip(ts, want[n % 3])), n
