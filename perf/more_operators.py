"""What a decode step and a training step need around the experts, as measured cases.

head_norm      root-mean-square norm of every query and key head with the position rotation behind it; and backward
linear_fp4     products of a few tokens with an NVFP4 or MXFP4 weight
decode_layer   the whole mixture-of-experts layer of a few tokens, with 16- or 32-bit expert weights

`own = False`: elementary torch operations; `own = True`: the package's kernels.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def _head(name, op, T, Hq, Hk, D, R, dtype, pairs, base, start):
    return dict(name=name, op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=R, dtype=dtype, pairs=pairs, base=base, start=start)


def _linear(name, T, N, K, fmt, dtype, f32_out=False):
    return dict(name=name, op="linear", T=T, N=N, K=K, fmt=fmt, dtype=dtype, f32_out=f32_out)


def _layer(name, T, H, E, I, k, dtype, shared, router, bias, base):
    return dict(name=name, op="layer", T=T, H=H, E=E, I=I, k=k, dtype=dtype, shared=shared, router=router, bias=bias, base=base)


def listed():
    return [
        # queries and keys of a decode step of four sequences, far into a long context
        _head("head norm decode", "head", 4, 32, 8, 128, 128, "bf16", False, 1e6, 130000),
        # the same for a 4096-token prompt
        _head("head norm prompt", "head", 4096, 64, 8, 128, 128, "bf16", False, 1e6, 0),
        # a ragged batch, heads of 96 of which 64 are rotated, neighbouring values paired
        _head("head norm ragged partial", "head", 1037, 24, 24, 96, 64, "f16", True, 1e4, 511),
        # training: gradients of queries, keys and both norm weights for a batch of 8192 tokens
        _head("head norm backward", "head_bwd", 8192, 32, 4, 128, 128, "bf16", False, 1e6, 0),
        # a projection of a decode step of four sequences
        _linear("linear decode", 4, 4096, 4096, "nvfp4", "bf16"),
        # a wide projection for sixteen tokens (four drafts of four sequences)
        _linear("linear verify", 16, 16384, 7168, "mxfp4", "bf16"),
        # logits of one sequence over a vocabulary of odd size, kept in 32 bits
        _linear("linear logits", 1, 100003, 4096, "nvfp4", "f16", True),
        # a batch of 64 sequences
        _linear("linear batch", 64, 7168, 2048, "nvfp4", "bf16"),
        # a small layer, one token: latency
        _layer("layer small", 1, 256, 8, 128, 2, "bf16", 0, "softmax", False, False),
        # a decode step of four sequences with a shared expert, added to the residual stream
        _layer("layer decode", 4, 4096, 128, 1536, 8, "bf16", 1536, "softmax", False, True),
        # sixteen tokens over a router with a bias
        _layer("layer verify", 16, 2048, 64, 1024, 6, "f16", 0, "sigmoid", True, False),
        # a 32-bit layer, three tokens
        _layer("layer f32", 3, 1024, 32, 768, 4, "f32", 0, "softmax", False, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("head", "head_bwd", "linear", "layer")}
    op = rng.choice(["head", "head_bwd", "linear", "linear", "layer", "layer"])
    if op in ("head", "head_bwd"):
        D = 16 * rng.randint(2, 16)
        c = dict(op=op, T=_log_int(rng, 1, 8192), Hq=_log_int(rng, 1, 64), Hk=_log_int(rng, 1, 16), D=D,
                 R=rng.choice([D, D, 16 * rng.randint(1, D // 16)]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                 pairs=rng.random() < 0.4, base=rng.choice([1e4, 5e5, 1e6]), start=rng.choice([0, 0, 1, 4095, 131072, 1000003]))
    elif op == "linear":
        c = dict(op=op, T=_log_int(rng, 1, 64), N=_log_int(rng, 16, 32768), K=128 * _log_int(rng, 2, 64),
                 fmt=rng.choice(["nvfp4", "nvfp4", "mxfp4"]), dtype=rng.choice(["bf16", "bf16", "f16"]), f32_out=rng.random() < 0.25)
    else:
        E = _log_int(rng, 4, 128)
        c = dict(op=op, T=_log_int(rng, 1, 16), H=64 * _log_int(rng, 4, 64), E=E, I=32 * _log_int(rng, 4, 48), k=rng.randint(1, min(8, E)),
                 dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), shared=rng.choice([0, 0, 32 * _log_int(rng, 4, 48)]),
                 router=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4, base=rng.random() < 0.5)
    while _cost(c) > most[op] and c["T"] > 1:
        c["T"] = c["T"] * 3 // 4
    while _cost(c) > most[op]:
        small = "N" if op == "linear" else "E"
        c[small] = max(c.get("k", 1), c[small] * 3 // 4)
    return c


def _cost(c):
    """Bytes that a pass moves, and for a layer those of all its weights too: they are made for every state."""
    b = work(c)["bytes"]
    return b + c["E"] * 3 * c["I"] * c["H"] * _size(c) if c["op"] == "layer" else b


def _size(c):
    return {"bf16": 2, "f16": 2, "f32": 4}[c["dtype"]]


def work(c):
    es, T = _size(c), c["T"]
    if c["op"] in ("head", "head_bwd"):
        n = T * (c["Hq"] + c["Hk"]) * c["D"]
        if c["op"] == "head":
            return {"bytes": 2 * n * es + 2 * c["D"] * es + 4 * T + 4 * c["R"], "flops": 8 * n}
        return {"bytes": 3 * n * es + 2 * c["D"] * (es + 4) + 4 * T + 4 * c["R"], "flops": 16 * n}
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        weight = N * K // 2 + N * K // (16 if c["fmt"] == "nvfp4" else 32)
        return {"bytes": weight + T * K * es + T * N * (4 if c["f32_out"] else es), "flops": 2 * T * N * K}
    H, E, I, k = c["H"], c["E"], c["I"], c["k"]
    touched = E * (1 - (1 - k / E) ** T)                    # experts that some token chooses, on average
    weights = 3 * H * (touched * I + c["shared"]) * es
    rows = T * H * es * (3 if c["base"] else 2) + 8 * T * k
    return {"bytes": int(weights + 4 * E * H + rows), "flops": 2 * T * H * (3 * (k * I + c["shared"]) + E)}


# ------------------------------------------------------------------ the inputs

def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _frequencies(c):
    """Radians a position, of the head's R / 2 planes of rotation."""
    return [c["base"] ** (-2.0 * i / c["R"]) for i in range(c["R"] // 2)]


def _turns(freqs):
    """The same as fractions of a turn in units of 2^-64, what a program keeps for head_norm."""
    u = [int(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freqs]
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in u], dtype=torch.int64, device="cuda")


def _quantise(w, fmt):
    """E2M1 codes (element 2i in the low half of byte i) and group scales of w [N][K]; NVFP4 with its tensor scale."""
    N, K = w.shape
    G = 16 if fmt == "nvfp4" else 32
    v = w.view(N, K // G, G)
    amax = v.abs().amax(2, keepdim=True)
    if fmt == "nvfp4":
        ts = w.abs().amax() / 2688
        scales = (amax / 6 / ts).to(E4M3)
        den = scales.float() * ts
        stored = scales.view(torch.uint8)
    else:
        ts = None
        stored = (torch.frexp(amax)[1] - 1 - 2 + 127).clamp(0, 254)
        den = torch.ldexp(torch.ones_like(amax), stored - 127)
        stored = stored.to(torch.uint8)
    q = torch.where(den == 0, 0.0, v / den)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    codes = torch.bucketize(q.abs(), borders).to(torch.uint8) | torch.where(q < 0, 8, 0).to(torch.uint8)
    codes = codes.view(N, K // 2, 2)
    return codes[:, :, 0] | (codes[:, :, 1] << 4), stored.view(N, K // G).contiguous(), ts


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 29)
    s, T, dt = dict(case=c), c["T"], DTYPES[c["dtype"]]
    if c["op"] in ("head", "head_bwd"):
        Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
        freqs = _frequencies(c)
        s["turns"], s["freqs"] = _turns(freqs), torch.tensor(freqs, dtype=torch.float64, device="cuda")
        # positions of several sequences behind one another, each from its own start
        length = max(1, T // 3)
        s["pos"] = (c["start"] + torch.arange(T, device="cuda") % length).to(torch.int32)
        s["qw"], s["kw"] = (_normal(g, (D,), torch.float32, 0.3).add_(1).to(dt) for _ in range(2))
        if c["op"] == "head":
            # queries and keys lie in the rows that one product of queries, keys and values gave
            qkv = _normal(g, (T, Hq + 2 * Hk, D), dt, 2.0)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
            s["out"] = dict(q=torch.empty(T, Hq, D, dtype=dt, device="cuda"), k=torch.empty(T, Hk, D, dtype=dt, device="cuda"))
        else:
            s["q"], s["k"] = _normal(g, (T, Hq, D), dt, 2.0), _normal(g, (T, Hk, D), dt, 2.0)
            s["gq"], s["gk"] = _normal(g, (T, Hq, D), dt), _normal(g, (T, Hk, D), dt)
            s["out"] = dict(grad_q=torch.empty_like(s["q"]), grad_k=torch.empty_like(s["k"]),
                            grad_qw=torch.empty(D, device="cuda"), grad_kw=torch.empty(D, device="cuda"))
        return s
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        # hidden states have a few channels far above the rest
        loud = 1 + 15 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = (_normal(g, (T, K), torch.float32) * loud).to(dt)
        s["codes"], s["scales"], s["ts"] = _quantise(_normal(g, (N, K), torch.float32, 0.02), c["fmt"])
        s["out"] = torch.empty(T, N, dtype=torch.float32 if c["f32_out"] else dt, device="cuda")
        return s
    H, E, I = c["H"], c["E"], c["I"]
    s["x"] = _normal(g, (T, H), dt)
    s["router"] = _normal(g, (E, H), torch.float32, H ** -0.5)
    s["bias"] = _normal(g, (E,), torch.float32, 0.5) if c["bias"] else None
    s["experts"] = (_normal(g, (E, I, H), dt, H ** -0.5), _normal(g, (E, I, H), dt, H ** -0.5), _normal(g, (E, H, I), dt, I ** -0.5))
    n = c["shared"]
    s["shared"] = (_normal(g, (n, H), dt, H ** -0.5), _normal(g, (n, H), dt, H ** -0.5), _normal(g, (H, n), dt, n ** -0.5)) if n else None
    s["base"] = _normal(g, (T, H), dt) if c["base"] else None
    s["out"] = dict(out=torch.empty(T, H, dtype=dt, device="cuda"), topk_ids=torch.empty(T, c["k"], dtype=torch.int32, device="cuda"),
                    topk_w=torch.empty(T, c["k"], device="cuda"))
    return s


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, c, back=False):
    """The first R values of every head rotated in their planes, by the angle or back."""
    R = c["R"]
    r = x[..., :R]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :R // 2], r[..., R // 2:])
    if back:
        sin = -sin
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if c["pairs"] else torch.cat([u, v], -1)
    return torch.cat([r, x[..., R:]], -1)


def _angles(s):
    a = s["pos"].double()[:, None] * s["freqs"]
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _plain_head(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        n = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w.float()
        return _rotate(n, cos, sin, c)

    return dict(q=one(s["q"], s["qw"]).to(s["q"].dtype), k=one(s["k"], s["kw"]).to(s["k"].dtype))


def _plain_head_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(g, x, w):
        g, x = _rotate(g.float(), cos, sin, c, back=True), x.float()
        rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * rstd
        gw = (g * n).double().sum((0, 1)).float()             # up to a million terms that nearly cancel
        g = g * w.float()
        return rstd * (g - n * (g * n).mean(-1, keepdim=True)), gw

    (gq, gqw), (gk, gkw) = one(s["gq"], s["q"], s["qw"]), one(s["gk"], s["k"], s["kw"])
    return dict(grad_q=gq.to(s["q"].dtype), grad_k=gk.to(s["k"].dtype), grad_qw=gqw, grad_kw=gkw)


def _plain_linear(s):
    codes, scales = s["codes"], s["scales"]
    N, groups = scales.shape
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    w = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).view(N, groups, -1)
    if s["ts"] is None:
        w = torch.ldexp(w, scales.int()[:, :, None] - 127)
    else:
        w = w * (scales.view(E4M3).float() * s["ts"])[:, :, None]
    return (s["x"].float() @ w.view(N, -1).T).to(s["out"].dtype)


def _plain_layer(s):
    c = s["case"]
    x, k = s["x"].float(), c["k"]
    logits = s["x"].double() @ s["router"].double().T          # 64 bits: neighbouring experts may be close
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    val, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    score = torch.exp(val - val[:, :1]) if c["router"] == "softmax" else 1 / (1 + torch.exp(-val))
    p = (score / score.sum(1, keepdim=True)).float()

    def ffn(x, gate, up, down):                                  # x [n][1][H], weights [n][.][.]
        a, b = x @ gate.float().mT, x @ up.float().mT
        return (a / (1 + torch.exp(-a)) * b) @ down.float().mT

    T, H = x.shape
    rows = x.repeat_interleave(k, 0)[:, None, :]
    at = ids.reshape(-1)
    gate, up, down = s["experts"]
    y = ffn(rows, gate[at], up[at], down[at]).view(T, k, H)
    out = (y * p[:, :, None]).sum(1)
    if s["shared"] is not None:
        out = out + ffn(x[None], *(w[None] for w in s["shared"]))[0]
    if s["base"] is not None:
        out = out + s["base"].float()
    return dict(out=out.to(s["x"].dtype), topk_ids=ids.to(torch.int32), topk_w=p)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import moe_routed_expert_router_gb300 as moe
        if op == "head":
            return moe.head_norm(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["turns"], interleaved=c["pairs"], eps=EPS, out=s["out"])
        if op == "head_bwd":
            return moe.head_norm_backward(s["gq"], s["gk"], s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["turns"],
                                          interleaved=c["pairs"], eps=EPS, out=s["out"])
        if op == "linear":
            return moe.linear_fp4(s["x"], moe.NvfpTensor(s["codes"], s["scales"], s["ts"]), out=s["out"])
        router = moe.ROUTER_SIGMOID if c["router"] == "sigmoid" else moe.ROUTER_SOFTMAX
        return moe.decode_layer(s["x"], s["router"], *s["experts"], c["k"], router_bias=s["bias"], router=router,
                                shared=s["shared"], base=s["base"], out=s["out"])
    if op == "head":
        return _plain_head(s)
    if op == "head_bwd":
        return _plain_head_bwd(s)
    return _plain_linear(s) if op == "linear" else _plain_layer(s)


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _exact_rotated(s, x, w):
    """x normed and turned as complex numbers: a plane's pair (a, b) is a + ib, times e^(i angle)."""
    c = s["case"]
    R = c["R"]
    n = x * torch.rsqrt(torch.einsum("thd,thd->th", x, x) / c["D"] + EPS)[:, :, None] * w
    z = n[..., :R].unflatten(-1, (R // 2, 2)) if c["pairs"] else n[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["pos"].double(), s["freqs"]))
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None, :])
    z = z.flatten(-2) if c["pairs"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, n[..., R:]], -1)


def _exact_head_bwd(s):
    def one(g, x, w):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        return torch.autograd.grad(_exact_rotated(s, x, w), (x, w), g.double())

    (gq, gqw), (gk, gkw) = one(s["gq"], s["q"], s["qw"]), one(s["gk"], s["k"], s["kw"])
    return dict(grad_q=gq, grad_k=gk, grad_qw=gqw, grad_kw=gkw)


def _exact_linear(s):
    N, K = s["case"]["N"], s["case"]["K"]
    x, out = s["x"].double(), []
    for n in range(0, N, 16384):
        codes = s["codes"][n:n + 16384].to(torch.int64)
        w = torch.empty(codes.shape[0], K, dtype=torch.float64, device="cuda")
        for half, nibble in ((0, codes & 15), (1, codes >> 4)):
            e, m = (nibble >> 1) & 3, (nibble & 1).double()
            v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
            w[:, half::2] = torch.where(nibble > 7, -v, v)
        sc = s["scales"][n:n + 16384]
        sc = torch.exp2(sc.double() - 127) if s["ts"] is None else sc.view(E4M3).double() * s["ts"].double()
        out.append(torch.einsum("tk,nk->tn", x, w * sc.repeat_interleave(K // sc.shape[1], 1)))
    return torch.cat(out, 1)


def _exact_layer(s):
    c = s["case"]
    x, T = s["x"].double(), c["T"]
    logits = torch.einsum("th,eh->te", x, s["router"].double()) + (0 if s["bias"] is None else s["bias"].double())
    val, ids = torch.topk(logits, c["k"], dim=1)
    p = torch.softmax(val, 1) if c["router"] == "softmax" else torch.sigmoid(val) / torch.sigmoid(val).sum(1, keepdim=True)

    def ffn(v, gate, up, down):
        return torch.einsum("hi,ti->th", down.double(), torch.nn.functional.silu(v @ gate.double().T) * (v @ up.double().T))

    out = torch.zeros_like(x) if s["base"] is None else s["base"].double().clone()
    if s["shared"] is not None:
        out += ffn(x, *s["shared"])
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        out[t] += p[t, j][:, None] * ffn(x[t], *(w[e] for w in s["experts"]))
    return dict(out=out, topk_ids=None, topk_w=p)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "head":
        return dict(q=_exact_rotated(s, s["q"].double(), s["qw"].double()), k=_exact_rotated(s, s["k"].double(), s["kw"].double()))
    if c["op"] == "head_bwd":
        return _exact_head_bwd(s)
    return _exact_linear(s) if c["op"] == "linear" else _exact_layer(s)
