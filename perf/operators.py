"""The operators of a mixture-of-experts layer's token path, as measured cases.

rms_norm       s = x + r, its root-mean-square norm, stored in the inputs' type or in 8 bits with scales; and backward
sort_pairs     (token, slot) pairs ordered by expert, every expert's segment padded to a multiple of rows
dispatch       token rows copied into that order (any type, with their scales); and backward
combine        expert rows weighted, added per token and brought back into token order; and backward

`own = False`: elementary torch operations; `own = True`: the package's kernels.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def _norm(name, T, H, dtype, quant, residual):
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, quant=quant, residual=residual)


def _moe(name, op, T, H, dtype, k, E, align, drop, **more):
    return dict(name=name, op=op, T=T, H=H, dtype=dtype, k=k, E=E, align=align, drop=drop, **more)


def listed():
    return [
        # the norm in front of a layer's products in a decode step of four sequences
        _norm("norm decode", 4, 4096, "bf16", "e4m3_128", True),
        # the same for a 4096-token prompt
        _norm("norm prompt", 4096, 7168, "bf16", "e4m3_128", True),
        # a ragged batch of a narrow model, microscaled output, a last block of 16 values
        _norm("norm ragged mx", 1037, 1840, "f16", "mxfp8", False),
        # training: gradients of input, residual and weight for a batch of 8192 tokens
        dict(name="norm backward", op="norm_bwd", T=8192, H=4096, dtype="bf16"),
        # routing of a decode step: 32 pairs, segments as they come
        dict(name="sort decode", op="sort", T=4, k=8, E=128, align=1, drop=0.0),
        # routing of a large training batch over 256 experts, segments padded to the product's 128-row tiles
        dict(name="sort batch", op="sort", T=16384, k=8, E=256, align=128, drop=0.05),
        # a decode step's rows to the experts
        _moe("dispatch decode", "dispatch", 4, 4096, "bf16", 8, 128, 1, 0.0),
        # a prompt's 8-bit rows with their scales, into 128-row tiles
        _moe("dispatch prompt 8 bit", "dispatch", 4096, 7168, "e4m3", 8, 256, 128, 0.0),
        # training: the gradient of the dispatched rows back to the tokens, some pairs dropped
        _moe("dispatch backward", "dispatch_bwd", 4093, 4096, "bf16", 8, 128, 16, 0.05),
        # a decode step's expert outputs with the shared expert's added
        _moe("combine decode", "combine", 4, 4096, "bf16", 8, 128, 1, 0.0, base=True),
        # a prompt's expert outputs back into token order
        _moe("combine prompt", "combine", 4096, 7168, "bf16", 8, 256, 128, 0.0, base=False),
        # training: gradients of the expert outputs and of the routing weights
        _moe("combine backward", "combine_bwd", 8192, 4096, "bf16", 8, 128, 128, 0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["norm", "norm", "norm_bwd", "sort", "dispatch", "dispatch_bwd", "combine", "combine_bwd"])
    c = dict(op=op, T=_log_int(rng, 1, 16384))
    if op != "sort":
        c["H"] = 16 * _log_int(rng, 16, 512)
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        c["quant"] = rng.choice(["none", "e4m3_128", "e4m3_row", "mxfp8"])
        c["residual"] = rng.random() < 0.6
    elif op != "norm_bwd":
        c["E"] = _log_int(rng, 4, 512)
        c["k"] = rng.randint(1, min(10, c["E"]))
        c["align"] = rng.choice([1, 1, 8, 16, 64, 128])
        c["drop"] = rng.choice([0.0, 0.0, 0.05, 0.5])
    if op == "dispatch" and rng.random() < 0.5:
        c["dtype"] = "e4m3"
    if op == "combine":
        c["base"] = rng.random() < 0.5
    while work(c)["bytes"] > most and c["T"] > 1:
        c["T"] = c["T"] * 3 // 4
    while work(c)["bytes"] > most and c["align"] > 1:
        c["align"] //= 2
    return c


def _rows(c):
    """Rows of the sorted layout: enough for any routing of the pairs."""
    P, A = c["T"] * c["k"], c["align"]
    return (P + min(c["E"], P) * (A - 1)) // A * A


def _scale_cols(quant, H):
    return {"e4m3_128": -(-H // 128), "e4m3_row": 1, "mxfp8": -(-H // 32)}[quant]


def work(c):
    op, T = c["op"], c["T"]
    es = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}.get(c.get("dtype"), 0)
    if op == "norm":
        H = c["H"]
        b = T * H * es * (3 if c["residual"] else 1) + H * es + 4 * T
        if c["quant"] == "none":
            b += T * H * es
        else:
            b += T * H + T * _scale_cols(c["quant"], H) * (1 if c["quant"] == "mxfp8" else 4)
        return {"bytes": b, "flops": 6 * T * H}
    if op == "norm_bwd":
        return {"bytes": 4 * T * c["H"] * es + 4 * T + c["H"] * (es + 4), "flops": 10 * T * c["H"]}
    P, R = T * c["k"], _rows(c)
    if op == "sort":
        return {"bytes": 8 * P + 4 * R + 4 * (c["E"] + 1), "flops": 0}
    H, kept = c["H"], int(P * (1 - c["drop"]))
    if op == "dispatch":
        row = H * es + (4 * _scale_cols("e4m3_128", H) if es == 1 else 0)
        return {"bytes": (T + R) * row + 4 * R, "flops": 0}
    if op == "dispatch_bwd":
        return {"bytes": (kept + T) * H * es + 4 * P, "flops": kept * H}
    if op == "combine":
        return {"bytes": (kept + T * (2 if c["base"] else 1)) * H * es + 8 * P, "flops": 2 * kept * H}
    return {"bytes": (T + kept + R) * H * es + 12 * P + 4 * R, "flops": 3 * kept * H}


# ------------------------------------------------------------------ the inputs

def _route(c, g):
    """Ids and weights of a skewed router (expert popularity ~ 1 / rank), some pairs dropped."""
    T, k, E = c["T"], c["k"], c["E"]
    dev = "cuda"
    rank = torch.randperm(E, generator=g, device=dev).float() + 1
    u = torch.rand(T, E, generator=g, device=dev).clamp_(1e-12, 1 - 1e-7)
    val, ids = torch.topk(-torch.log(rank) - torch.log(-torch.log(u)), k, dim=1)
    weights = torch.softmax(val, dim=1)
    if c["drop"]:
        gone = torch.rand(T, k, generator=g, device=dev) < c["drop"]
        if T > 1:
            gone[T // 2] = True           # a token none of whose pairs is kept
        ids = torch.where(gone, -1, ids)
    return ids.to(torch.int32).contiguous(), weights.contiguous()


def _order(ids, E, align, R):
    """offsets, rows, inv of the sorted layout."""
    P, dev = ids.numel(), ids.device
    e = ids.reshape(-1).long()
    e = torch.where((e < 0) | (e >= E), E, e)                  # dropped pairs sort last
    count = torch.zeros(E + 1, dtype=torch.int64, device=dev).scatter_add_(0, e, torch.ones_like(e))
    start = torch.cumsum(count, 0) - count                     # of every expert, unpadded
    padded = torch.cumsum((count[:E] + align - 1) // align * align, 0)
    offsets = torch.cat([padded.new_zeros(1), padded])
    perm = torch.argsort(e, stable=True)
    es = e[perm]
    row = offsets[es] + torch.arange(P, device=dev) - start[es]
    row = torch.where(es == E, -1, row)
    inv = torch.empty_like(e)
    inv[perm] = row
    rows = torch.full((R + 1,), -1, dtype=torch.int64, device=dev)
    rows[torch.where(row < 0, R, row)] = perm                  # dropped ones land in the spare place
    i32 = torch.int32
    return offsets.to(i32), rows[:R].to(i32), inv.to(i32).reshape(ids.shape)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    s, T, op = dict(case=c), c["T"], c["op"]
    if op in ("norm", "norm_bwd"):
        H, dt = c["H"], DTYPES[c["dtype"]]
        # hidden states have a few channels far above the rest
        loud = 1 + 15 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s["w"] = _normal(g, (H,), torch.float32, 0.2).add_(1).to(dt)
        if op == "norm":
            s["x"] = _normal(g, (T, H), dt)
            s["r"] = (_normal(g, (T, H), torch.float32, 2.0) * loud).to(dt) if c["residual"] else None
            out = dict(rstd=torch.empty(T, device="cuda"))
            if c["residual"]:
                out["sum"] = torch.empty(T, H, dtype=dt, device="cuda")
            if c["quant"] == "none":
                out["y"] = torch.empty(T, H, dtype=dt, device="cuda")
            else:
                out["q"] = torch.empty(T, H, dtype=E4M3, device="cuda")
                out["scales"] = torch.empty(T, _scale_cols(c["quant"], H), device="cuda",
                                            dtype=torch.float8_e8m0fnu if c["quant"] == "mxfp8" else torch.float32)
        else:
            s["s"] = (_normal(g, (T, H), torch.float32, 2.0) * loud).to(dt)
            s["rstd"] = (s["s"].double().square().mean(1) + EPS).rsqrt().float()
            s["gy"] = _normal(g, (T, H), dt)
            s["gs"] = _normal(g, (T, H), dt, 0.5)
            out = dict(grad_sum=torch.empty(T, H, dtype=dt, device="cuda"), grad_w=torch.empty(H, device="cuda"))
        s["out"] = out
        return s
    ids, weights = _route(c, g)
    R, P = _rows(c), T * c["k"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "sort":
        s["ids"] = ids
        s["out"] = dict(expert_offsets=torch.empty(c["E"] + 1, **i32), sorted_rows=torch.empty(R, **i32),
                        pair_rows=torch.empty(T, c["k"], **i32))
        return s
    offsets, rows, inv = _order(ids, c["E"], c["align"], R)
    s["order"] = dict(expert_offsets=offsets, sorted_rows=rows, pair_rows=inv)
    H = c["H"]
    dt = DTYPES.get(c["dtype"], E4M3)
    if op == "dispatch":
        s["x"] = _normal(g, (T, H), torch.float32, 100.0 if dt == E4M3 else 1.0).clamp_(-448, 448).to(dt)
        s["out"] = dict(rows=torch.empty(R, H, dtype=dt, device="cuda"))
        if dt == E4M3:
            n = _scale_cols("e4m3_128", H)
            s["scales"] = torch.rand(T, n, generator=g, device="cuda") + 0.01
            s["out"]["scales"] = torch.empty(R, n, device="cuda")
        return s
    # rows that no pair holds were never written by the expert's product: whatever is there is not to be read
    y = _normal(g, (R, H), dt)
    y[rows < 0] = float("nan")
    s["y"], s["w"] = y, weights
    if op == "combine_bwd":
        s["go"] = _normal(g, (T, H), dt)
        s["out"] = dict(grad_y=torch.empty(R, H, dtype=dt, device="cuda"), grad_w=torch.empty(T, c["k"], device="cuda"))
    else:
        s["base"] = _normal(g, (T, H), dt) if c.get("base") else None
        s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _groups(n, quant):
    """n [T][H] as [T][groups][values], the last group filled up with zeros."""
    T, H = n.shape
    G = {"e4m3_128": 128, "e4m3_row": H, "mxfp8": 32}[quant]
    cols = -(-H // G)
    if cols * G != H:
        n = torch.cat([n, n.new_zeros(T, cols * G - H)], dim=1)
    return n.reshape(T, cols, G)


def _plain_norm(s):
    c, out = s["case"], {}
    x = s["x"].float()
    if c["residual"]:
        out["sum"] = (x + s["r"].float()).to(s["x"].dtype)
        x = out["sum"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    out["rstd"] = rstd[:, 0]
    n = x * rstd * s["w"].float()
    if c["quant"] == "none":
        out["y"] = n.to(s["x"].dtype)
        return out
    T, H = n.shape
    v = _groups(n, c["quant"])
    amax = v.abs().amax(2, keepdim=True)
    if c["quant"] == "mxfp8":
        byte = (torch.frexp(amax)[1] - 1 - 8 + 127).clamp(0, 254)
        byte = torch.where(amax == 0, 0, byte)
        q = v * torch.ldexp(torch.ones_like(amax), 127 - byte)
        out["scales"] = byte[:, :, 0].to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        amax = amax.clamp(min=2.0 ** -100)
        q = v * (448.0 / amax)
        out["scales"] = amax[:, :, 0] / 448.0
    out["q"] = q.clamp(-448, 448).reshape(T, -1)[:, :H].contiguous().to(E4M3)
    return out


def _plain_norm_bwd(s):
    gy, x, rstd = s["gy"].float(), s["s"].float(), s["rstd"][:, None]
    n = x * rstd
    g = gy * s["w"].float()
    gs = rstd * (g - n * (g * n).mean(1, keepdim=True)) + s["gs"].float()
    return dict(grad_sum=gs.to(s["s"].dtype), grad_w=(gy * n).sum(0))


def _plain_dispatch(s):
    rows = s["order"]["sorted_rows"].long()
    t = torch.where(rows < 0, s["case"]["T"], rows // s["case"]["k"])

    def gather(x):   # bytes, and a row of zeros for the rows without a pair
        b = x.view(torch.uint8)
        return torch.cat([b, b.new_zeros(1, b.shape[1])])[t].view(x.dtype)

    out = dict(rows=gather(s["x"]))
    if "scales" in s:
        out["scales"] = gather(s["scales"])
    return out


def _pair_rows(s):
    """The pairs' rows of y in fp32, [T][k][H], zero where a pair is dropped."""
    inv = s["order"]["pair_rows"].long()
    y = s["y"][inv.clamp(min=0)].float()
    return torch.where((inv < 0)[:, :, None], 0.0, y)


def _plain_combine(s, weights, base):
    y = _pair_rows(s)
    acc = (y if weights is None else y * weights[:, :, None]).sum(1)
    if base is not None:
        acc = acc + base.float()
    return acc.to(s["y"].dtype)


def _plain_combine_bwd(s):
    c = s["case"]
    go = s["go"].float()
    rows = s["order"]["sorted_rows"].long()
    p = rows.clamp(min=0)
    gy = go[p // c["k"]] * s["w"].reshape(-1)[p][:, None]
    gy = torch.where((rows < 0)[:, None], 0.0, gy).to(s["y"].dtype)
    return dict(grad_y=gy, grad_w=(_pair_rows(s) * go[:, None, :]).sum(2))


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import moe_routed_expert_router_gb300 as moe
        if op == "norm":
            quant = {"none": moe.QUANT_NONE, "e4m3_128": moe.QUANT_E4M3_128, "e4m3_row": moe.QUANT_E4M3_ROW,
                     "mxfp8": moe.QUANT_MXFP8}[c["quant"]]
            return moe.rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, quant=quant, out=s["out"])
        if op == "norm_bwd":
            return moe.rms_norm_backward(s["gy"], s["s"], s["w"], s["rstd"], grad_sum=s["gs"], out=s["out"])
        if op == "sort":
            return moe.sort_pairs(s["ids"], c["E"], align=c["align"], out=s["out"])
        if op == "dispatch":
            return moe.dispatch(s["x"], s["order"], scales=s.get("scales"), out=s["out"])
        if op == "dispatch_bwd":
            return moe.dispatch_backward(s["y"], s["order"], out=s["out"])
        if op == "combine":
            return moe.combine(s["y"], s["order"], s["w"], base=s["base"], out=s["out"])
        return moe.combine_backward(s["go"], s["y"], s["order"], s["w"], out=s["out"])
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "sort":
        offsets, rows, inv = _order(s["ids"], c["E"], c["align"], _rows(c))
        return dict(expert_offsets=offsets, sorted_rows=rows, pair_rows=inv)
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "dispatch_bwd":
        return _plain_combine(s, None, None)
    if op == "combine":
        return _plain_combine(s, s["w"], s["base"])
    return _plain_combine_bwd(s)


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _e4m3_64(v):
    """Round to nearest even onto the E4M3 grid: 3 fraction bits, exponents from -6, at most 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_norm(s):
    c, out = s["case"], {}
    x = s["x"].double()
    if c["residual"]:
        out["sum"] = x + s["r"].double()
        x = out["sum"].to(s["x"].dtype).double()      # the norm is the stored sum's
    T, H = x.shape
    rstd = torch.rsqrt(torch.einsum("th,th->t", x, x) / H + EPS)
    out["rstd"] = rstd
    n = torch.einsum("th,t,h->th", x, rstd, s["w"].double())
    if c["quant"] == "none":
        out["y"] = n
        return out
    G = {"e4m3_128": 128, "e4m3_row": H, "mxfp8": 32}[c["quant"]]
    scales = torch.empty(T, -(-H // G), dtype=torch.float64, device=x.device)
    q = torch.empty_like(n)
    for i in range(scales.shape[1]):
        v = n[:, i * G:(i + 1) * G]
        a = v.abs().max(1).values
        if c["quant"] == "mxfp8":
            scales[:, i] = torch.exp2((torch.floor(torch.log2(a)) - 8).clamp(-127, 127))
        else:
            scales[:, i] = a.clamp(min=2.0 ** -100) / 448
        q[:, i * G:(i + 1) * G] = _e4m3_64(v / scales[:, i:i + 1])
    out["q"], out["scales"] = q, scales
    return out


def _exact_norm_bwd(s):
    x, w, gy = s["s"].double(), s["w"].double(), s["gy"].double()
    r = s["rstd"].double()
    dot = torch.einsum("th,th,h->t", gy, x, w) / x.shape[1]
    gx = torch.einsum("t,th,h->th", r, gy, w) - torch.einsum("t,th->th", r ** 3 * dot, x) + s["gs"].double()
    return dict(grad_sum=gx, grad_w=torch.einsum("th,th,t->h", gy, x, r))


def exact(c, seed):
    if c["op"] in ("sort", "dispatch"):
        return None                                   # whole numbers and copies
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(s)
    if c["op"] == "norm_bwd":
        return _exact_norm_bwd(s)
    T, H, k = c["T"], c["H"], c["k"]
    inv = s["order"]["pair_rows"].long()
    y = s["y"]
    if c["op"] == "combine_bwd":
        gy = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
        gw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        go = s["go"].double()
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            gy[inv[t, j]] = go[t] * s["w"][t, j].double()[:, None]
            gw[t, j] = (go[t] * y[inv[t, j]].double()).sum(1)
        return dict(grad_y=gy, grad_w=gw)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(inv[:, j] >= 0)[:, 0]
        v = y[inv[t, j]].double()
        out[t] += v * s["w"][t, j].double()[:, None] if c["op"] == "combine" else v
    return out + s["base"].double() if c["op"] == "combine" and s["base"] is not None else out
