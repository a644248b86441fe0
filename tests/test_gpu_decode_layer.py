"""decode_layer against the layer in 64 bits.

Tolerances count roundings, u = 2^-24.  Logits: a lane adds H / 32 products in turn, five levels join the lanes and one
adds the bias, so they are off by less than (H / 32 + 8) u of the sum of magnitudes; the weights, whose relative error is
at most twice that of a logit and ten roundings, follow.  A product of K values: K / 64 additions a lane half, six to
join them.  h = w silu(g) u moves with g by at most 1.1 |u| and with u by |silu(g)|, plus ten roundings."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Layer:
    def __init__(self, T, H, E, I, k, dtype, shared=0, bias=False, base=False, router=moe.ROUTER_SOFTMAX, renorm=True, rdt=torch.float32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DTYPES[dtype]

        def normal(*shape, std=1.0, to=dt):
            return (std * torch.randn(shape, generator=g, device="cuda")).to(to)
        self.T, self.k, self.dt, self.router, self.renorm = T, k, dt, router, renorm
        self.x = normal(T, H)
        self.rw = normal(E, H, std=H ** -0.5, to=rdt)
        self.bias = normal(E, to=torch.float32) if bias else None
        self.gate, self.up, self.down = normal(E, I, H, std=H ** -0.5), normal(E, I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5)
        self.shared = (normal(shared, H, std=H ** -0.5), normal(shared, H, std=H ** -0.5), normal(H, shared, std=shared ** -0.5)) if shared else None
        self.base = normal(T, H) if base else None

    def run(self, **kw):
        return moe.decode_layer(self.x, self.rw, self.gate, self.up, self.down, self.k, router_bias=self.bias, router=self.router,
                                renormalize=self.renorm, shared=self.shared, base=self.base, **kw)


def dots(x, w):
    """x [n][K] times w [N][K] in 64 bits, and the error allowed."""
    K = x.shape[1]
    return x @ w.T, (K / 64 + 8) * U * (x.abs() @ w.abs().T)


def ffn(x, gate, up, down, p, dp):
    """p * FFN(x) in 64 bits and the error allowed; dp: that of p."""
    gate, up, down = gate.double(), up.double(), down.double()
    (g, eg), (u, eu) = dots(x, gate), dots(x, up)
    silu = g * torch.sigmoid(g)
    h = silu * u
    eh = 1.1 * u.abs() * eg + silu.abs() * eu + 10 * U * h.abs()
    y, ey = dots(p * h, down)
    return y, ey + (p * eh + dp * h.abs()) @ down.abs().T


def check(L, got):
    x = L.x.double()
    T, H = x.shape
    E = L.rw.shape[0]
    logits = x @ L.rw.double().T
    el = (H / 32 + 8) * U * (x.abs() @ L.rw.double().abs().T) + U
    if L.bias is not None:
        logits = logits + L.bias.double()
        el = el + U * logits.abs()
    ids = got["topk_ids"].long()
    assert ids.dtype == torch.int64 and (ids >= 0).all() and (ids < E).all()
    for t in range(T):
        assert len(set(ids[t].tolist())) == L.k
    val, e = logits.gather(1, ids), el.gather(1, ids)
    assert (val[:, :-1] + e[:, :-1] >= val[:, 1:] - e[:, 1:]).all()          # by decreasing logit
    left = logits.scatter(1, ids, float("-inf"))
    assert (val[:, -1:] + e[:, -1:] + el >= left).all()                       # and nothing larger is left out
    if L.router == moe.ROUTER_SOFTMAX:
        m = logits.amax(1, keepdim=True)
        num = torch.exp(val - m)
        den = num.sum(1, keepdim=True) if L.renorm else torch.exp(logits - m).sum(1, keepdim=True)
    else:
        num = torch.sigmoid(val)
        den = num.sum(1, keepdim=True) if L.renorm else torch.ones_like(num[:, :1])
    p = num / den
    ep = p * (4 * el.amax(1, keepdim=True) + (10 + E / 32) * U)
    assert ((got["topk_w"].double() - p).abs() <= ep).all()
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    for ex in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == ex, as_tuple=True)
        a, b = ffn(x[t], L.gate[ex], L.up[ex], L.down[ex], p[t, j][:, None], ep[t, j][:, None])
        y[t] += a
        tol[t] += b + 40 * U * a.abs()
    if L.shared is not None:
        one = torch.ones(T, 1, dtype=torch.float64, device="cuda")
        a, b = ffn(x, *L.shared, one, 0 * one)
        y, tol = y + a, tol + b + 40 * U * a.abs()
    if L.base is not None:
        y = y + L.base.double()
        tol = tol + U * y.abs()
    half = torch.finfo(L.dt).eps / 2
    least = torch.finfo(L.dt).smallest_normal * half
    assert ((got["out"].double() - y).abs() <= tol * (1 + half) + y.abs() * half + least).all()


# one token to sixteen; experts with one to sixteen tokens; widths below a warp's step, odd and ragged; fewer rows than
# blocks; every expert chosen; many experts
CASES = [
    dict(T=1, H=8, E=1, I=8, k=1), dict(T=1, H=256, E=8, I=128, k=2), dict(T=4, H=512, E=16, I=256, k=4, shared=128, base=True),
    dict(T=16, H=264, E=4, I=136, k=4, shared=72), dict(T=16, H=1000, E=40, I=328, k=6, bias=True),
    dict(T=7, H=520, E=3, I=1032, k=2, base=True), dict(T=3, H=2048, E=32, I=768, k=8), dict(T=2, H=5128, E=6, I=64, k=3, shared=2056),
    dict(T=16, H=64, E=1024, I=16, k=32), dict(T=9, H=128, E=33, I=40, k=32, shared=8, bias=True, base=True),
    dict(T=5, H=16384, E=2, I=24, k=2), dict(T=1, H=24, E=2, I=16384, k=1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_against_64_bits(case, dtype):
    for i, (router, renorm) in enumerate([(moe.ROUTER_SOFTMAX, True), (moe.ROUTER_SIGMOID, True), (moe.ROUTER_SOFTMAX, False), (moe.ROUTER_SIGMOID, False)]):
        if i and case["H"] > 1000:
            continue
        L = Layer(**case, dtype=dtype, router=router, renorm=renorm, rdt=torch.bfloat16 if i % 2 else torch.float32, seed=i)
        got = L.run()
        check(L, got)
        again = L.run()
        for name in got:
            assert torch.equal(got[name], again[name])               # a fixed order of sums


@pytest.mark.parametrize("router,renorm,bias,rdt", [(moe.ROUTER_SOFTMAX, True, False, torch.float32), (moe.ROUTER_SIGMOID, True, True, torch.bfloat16),
                                                    (moe.ROUTER_SOFTMAX, False, True, torch.float32), (moe.ROUTER_SIGMOID, False, False, torch.bfloat16)])
@pytest.mark.parametrize("T,H,E,k", [(1, 256, 8, 2), (4, 4096, 128, 8), (16, 512, 1024, 32), (16, 7168, 256, 8)])
def test_ids_and_weights_are_the_routers(T, H, E, k, router, renorm, bias, rdt):
    """Bit for bit what Plan.route gives."""
    L = Layer(T, H, E, 8, k, "bf16", bias=bias, router=router, renorm=renorm, rdt=rdt, seed=T)
    got = L.run()
    with moe.Plan(H, 128, E, k, T, router=router, renormalize=renorm, router_dtype=moe.ROUTER_BF16 if rdt is torch.bfloat16 else moe.ROUTER_F32) as plan:
        want = plan.route(L.x, L.rw, L.bias)
        assert plan.sync_status() == moe.OK
    assert torch.equal(got["topk_ids"], want["topk_ids"]) and torch.equal(got["topk_w"], want["topk_w"])


def test_ties_go_to_the_lower_id():
    L = Layer(3, 256, 12, 64, 5, "bf16", seed=1)
    L.rw[:] = L.rw[0]
    got = L.run()
    assert (got["topk_ids"] == torch.arange(5, device="cuda")).all() and (got["topk_w"] - 0.2).abs().max() < 1e-6


def test_tokens_that_are_not_finite_stay_alone():
    L = Layer(5, 512, 16, 128, 4, "bf16", shared=64, seed=2)
    good = L.run()
    L.x[1, 7], L.x[3, 100] = float("nan"), float("inf")
    bad = L.run()
    for name in good:
        assert torch.equal(good[name][[0, 2, 4]], bad[name][[0, 2, 4]])
    assert bad["out"][1].isnan().all()
    assert bad["topk_ids"][1].tolist() == [0, 1, 2, 3] and bad["topk_w"][1].isnan().all()      # NaN logits tie
    assert not bad["out"][3].isfinite().any()


def test_out_over_x_and_over_base():
    L = Layer(6, 768, 8, 96, 3, "f16", base=True, seed=3)
    want = L.run()["out"].clone()
    ids, w = torch.empty(6, 3, dtype=torch.int32, device="cuda"), torch.empty(6, 3, device="cuda")
    x, base = L.x.clone(), L.base.clone()
    L.run(out=dict(out=L.base, topk_ids=ids, topk_w=w))
    assert torch.equal(L.base, want)
    L.x, L.base = x, base
    L.run(out=dict(out=L.x, topk_ids=ids, topk_w=w))
    assert torch.equal(L.x, want)


def test_no_tokens():
    L = Layer(2, 64, 4, 32, 2, "f32")
    L.x = L.x[:0]
    got = L.run()
    assert got["out"].shape == (0, 64) and got["topk_ids"].shape == (0, 2)


def test_experts_past_four_gigabytes():
    """Offsets beyond 32 bits: the last experts of 5 GB a matrix, all others NaN."""
    T, H, E, I, k = 3, 4096, 512, 1280, 2
    L = Layer(T, H, 2, I, k, "bf16", seed=4)
    big = Layer.__new__(Layer)
    big.__dict__.update(L.__dict__)
    for name in ("gate", "up", "down"):
        w = getattr(L, name)
        full = torch.full((E, *w.shape[1:]), float("nan"), dtype=w.dtype, device="cuda")
        full[-2:] = w
        setattr(big, name, full)
    big.rw = torch.zeros(E, H, device="cuda")
    big.rw[-2:] = L.rw
    big.bias = torch.full((E,), -100.0, device="cuda")
    big.bias[-2:] = 0
    L.bias = torch.zeros(2, device="cuda")
    got, want = big.run(), L.run()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["topk_ids"], want["topk_ids"] + E - 2)


def test_captured_replayed_and_beside_another_stream():
    L, M = Layer(4, 1024, 16, 256, 4, "bf16", shared=128, seed=5), Layer(16, 512, 32, 512, 6, "bf16", seed=6)
    L.run(), M.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = L.run(), M.run()
        c = moe.decode_layer(a["out"], L.rw, L.gate, L.up, L.down, 4)          # on the result of the call before
    side = torch.cuda.Stream()
    for seed in (7, 8):
        L.x.copy_(torch.randn(L.x.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        one, two = L.run(stream=side), M.run()                                 # at the same time
        torch.cuda.synchronize()
        for got, want in ((a, one), (b, two)):
            for name in got:
                assert torch.equal(got[name], want[name])
        check(L, a)
        assert torch.equal(c["out"], moe.decode_layer(a["out"], L.rw, L.gate, L.up, L.down, 4)["out"])


def test_many_calls_at_once():
    """Layers on three streams beside products that hold the card: each call's blocks wait inside for others of its own,
    and have to finish whatever else keeps them from running together."""
    layers = [Layer(4, 2048, 16, 256, 4, "bf16", shared=128, seed=9), Layer(16, 1024, 32, 128, 6, "f16", seed=10), Layer(1, 4096, 8, 512, 2, "f32", seed=11)]
    want = [L.run() for L in layers]
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    streams, big, got = [torch.cuda.Stream() for _ in layers], torch.cuda.Stream(), []
    for _ in range(12):
        with torch.cuda.stream(big):
            for _ in range(4):
                torch.mm(a, a)
        got += [L.run(stream=s) for L, s in zip(layers, streams)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for name in out:
            assert torch.equal(out[name], want[i % 3][name])


def test_workspaces_of_calls_behind_one_another():
    """Calls of different sizes, nothing waiting between them: each has the memory of the one before."""
    layers = [Layer(T, 512, 24, 64 * (1 + T % 3), 4, "bf16", base=True, seed=20 + T) for T in (16, 1, 7, 2, 12)]
    want = [L.run()["out"].clone() for L in layers]
    got = [L.run()["out"] for _ in range(6) for L in layers]
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 5])
