"""linear_fp4 against the product in 64 bits.

Tolerances count roundings, u = 2^-24.  A weight value enters as code times scale, exact in f16 (NVFP4), or its scale
multiplies the fp32 sum of 32 products (MXFP4, one rounding).  The products are exact in fp32; the sums run over K in any
order, the matrix unit's own included, for which two steps (4 u) an addition of 16 products are allowed: with K / 16
additions a chain, and the join of eight chains, the sum is off by less than (K / 4 + 16) u of the sum of magnitudes.
bf16 rows are off by 2^-32 of their largest finite value."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def weight64(w):
    """The weight's values without its tensor scale, [N][K] in 64 bits."""
    codes, scales = w.codes.reshape(-1, w.codes.shape[-1]).long(), w.scales.reshape(-1, w.scales.shape[-1])
    v = VALUES.to(codes.device)[torch.stack([codes & 15, codes >> 4], -1)].flatten(1)
    if w.ts is None:
        s = torch.exp2(scales.double() - 127)
        s = torch.where(scales == 255, float("nan"), s)
    else:
        s = scales.view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(v.shape[1] // s.shape[1], 1)


def a_weight(N, K, fmt, seed=0):
    """Codes of every value and scales over their whole ordinary range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "nvfp4":
        scales = torch.randint(0, 127, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)     # 0 to 448, with subnormals
        return moe.NvfpTensor(codes, scales, torch.tensor([0.0173], device="cuda"))
    return moe.NvfpTensor(codes, torch.randint(97, 157, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8), None)


def rows(T, K, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, generator=g, device="cuda")
    x[:, ::97] *= 50
    x[:, 5::89] *= 2.0 ** -12
    return x.to(dt)


def check(out, x, w):
    m = weight64(w)
    ts = 1.0 if w.ts is None else w.ts.double().item()
    x = x.double()
    y, size = (x @ m.T) * ts, (x.abs() @ m.abs().T) * abs(ts)
    K = x.shape[1]
    tol = (K / 4 + 20) * U * size + 2.0 ** -32 * x.abs().amax(1, keepdim=True) * m.abs().sum(1) * abs(ts)
    half = torch.finfo(out.dtype).eps / 2
    least = torch.finfo(out.dtype).smallest_normal * half
    assert ((out.double() - y).abs() <= tol * (1 + half) + y.abs() * half + least).all()


# tokens of every tile width and its borders, odd numbers of rows, K of one stage, of partial stages, of fewer stages than
# warps, of several rounds of the ring and of several tiles a block
SHAPES = [(1, 1, 128), (1, 16, 256), (3, 17, 384), (8, 130, 512), (9, 33, 640), (16, 100, 1024), (17, 257, 1920), (31, 64, 2048),
          (32, 48, 4096), (33, 1000, 2176), (64, 515, 7168), (65, 40, 512), (130, 96, 1152), (2, 20011, 4096), (5, 9000, 8192), (1, 3, 65536)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_against_64_bits(T, N, K, dt, fmt):
    x, w = rows(T, K, dt, T + K), a_weight(N, K, fmt, N + K)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    assert out.dtype is F32 and out.shape == (T, N)
    check(out, x, w)
    same = moe.linear_fp4(x, w)
    assert same.dtype is dt
    assert torch.equal(same, out.to(dt))                          # one rounding of the same sums


@pytest.mark.parametrize("T", [1, 8, 16, 64])
def test_quantised_weights_of_the_packages_own(T):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = 0.02 * torch.randn(272, 1024, generator=g, device="cuda")
    x = rows(T, 1024, BF, 2)
    check(moe.linear_fp4(x, moe.quantize_nvfp4(w)), x, moe.quantize_nvfp4(w))
    check(moe.linear_fp4(x, moe.quantize_mxfp4(w)), x, moe.quantize_mxfp4(w))


def test_a_token_does_not_depend_on_the_others():
    """Any batch gives the bits of the same tile width's others: rows behind the last one are not read."""
    w = a_weight(200, 1024, "nvfp4")
    x = rows(8, 1024, BF)
    all8 = moe.linear_fp4(x, w, out_dtype=F32)
    for T in range(1, 8):
        assert torch.equal(moe.linear_fp4(x[:T], w, out_dtype=F32), all8[:T])
    x[3] = float("nan")
    x[5, 17] = float("inf")
    bad = moe.linear_fp4(x, w, out_dtype=F32)
    keep = [0, 1, 2, 4, 6, 7]
    assert torch.equal(bad[keep], all8[keep]) and bad[3].isnan().all()
    m = weight64(w)
    want = x[5].double()[None] * m                                # inf times a zero is NaN, as in any arithmetic
    assert torch.equal(bad[5].isnan(), want.sum(1).isnan())
    fine = ~bad[5].isnan()
    assert torch.equal(bad[5][fine], want.sum(1)[fine].float())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_strided_rows_and_sizes_of_rows(fmt):
    T, K = 6, 768
    store = torch.full((T, 1000), float("nan"), dtype=BF, device="cuda")
    x = store[:, 8:8 + K]
    x.copy_(rows(T, K, BF, 4))
    w = a_weight(70, K, fmt)
    assert torch.equal(moe.linear_fp4(x, w), moe.linear_fp4(x.contiguous(), w))
    x16 = torch.full((T, 1000), float("nan"), dtype=F16, device="cuda")[:, 16:16 + K]
    x16.copy_(rows(T, K, F16, 4))
    assert torch.equal(moe.linear_fp4(x16, w), moe.linear_fp4(x16.contiguous(), w))


@pytest.mark.parametrize("exponent", [-120, -60, 0, 60, 115])
def test_rows_of_any_size(exponent):
    """bf16 rows from the smallest to the largest magnitudes, one of zeros, and one of both ends."""
    K = 512
    w = moe.NvfpTensor(a_weight(40, K, "nvfp4").codes, torch.full((40, K // 16), 0x08, dtype=torch.uint8, device="cuda"),
                       torch.tensor([1.0], device="cuda"))        # scales of 2^-6
    x = (rows(4, K, F32, 7).double() * 2.0 ** exponent).to(BF)
    x[1] = 0
    x[2, ::2] = 2.0 ** -126
    out = moe.linear_fp4(x, w, out_dtype=F32)
    check(out, x, w)
    assert (out[1] == 0).all()


def test_mxfp4_scales_of_any_size():
    """Block scales far outside f16's range, each block's share kept: rows of one scale, and rows of both ends."""
    K, N = 256, 48
    w = a_weight(N, K, "mxfp4")
    w.scales[:16] = 30
    w.scales[16:32] = 215
    w.scales[32:, ::2], w.scales[32:, 1::2] = 40, 200
    x = rows(5, K, BF, 9)
    check(moe.linear_fp4(x, w, out_dtype=F32), x, w)
    only = x.clone()
    only.view(5, K // 64, 2, 32)[:, :, 1] = 0                     # the small blocks alone
    check(moe.linear_fp4(only, w, out_dtype=F32), only, w)
    w.scales[7, 3] = 255                                          # NaN
    bad = moe.linear_fp4(x, w, out_dtype=F32)
    assert bad[:, 7].isnan().all() and bad.isnan().sum() == 5


def test_no_tokens():
    w = a_weight(16, 128, "nvfp4")
    assert moe.linear_fp4(torch.empty(0, 128, dtype=BF, device="cuda"), w).shape == (0, 16)


def test_weights_past_four_gigabytes():
    """Code offsets beyond 32 bits: the last rows of a weight of 4.5 GB."""
    N, K = (1 << 32) // 32768 + 5000, 65536
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda")          # 1
    tail = a_weight(300, K, "nvfp4")
    codes[-300:], scales[-300:] = tail.codes, tail.scales
    ts = torch.tensor([0.0173], device="cuda")
    x = rows(3, K, F16, 5)
    out = moe.linear_fp4(x, moe.NvfpTensor(codes, scales, ts), out_dtype=F32)
    assert (out[:, :-300] == 0).all()
    check(out[:, -300:], x, moe.NvfpTensor(tail.codes, tail.scales, ts))


def test_captured_and_replayed_beside_other_calls():
    """Graphs and streams: the workspace of a call is its own, and a weight written by the call before is read as written."""
    K, N = 2048, 512
    x, w32 = rows(4, K, BF, 11), 0.02 * torch.randn(N, K, device="cuda")
    w = moe.quantize_nvfp4(w32)
    moe.linear_fp4(x, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.quantize_nvfp4(w32, out=w)
        one = moe.linear_fp4(x, w)
        two = moe.linear_fp4(x * 2, w)
    side = torch.cuda.Stream()
    for seed in (12, 13):
        x.copy_(rows(4, K, BF, seed))
        w32.copy_(0.02 * torch.randn(N, K, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        check(one, x, w)
        assert torch.equal(two, one * 2)
        got = [moe.linear_fp4(x, w, stream=side), moe.linear_fp4(x, w)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], one) and torch.equal(got[1], one)
