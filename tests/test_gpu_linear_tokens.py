"""linear_fp4 with more tokens than eight and large weights: the product on the block-scaled tensor cores, which takes
tokens as integers in octal digits.  The tolerance of the sums is test_gpu_linear's; a value is off by half a step of its
scale block's integers, at most 2^-22 of the block's largest value, or for NVFP4 2^-30 of the token's where that is more."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_linear import BF, F16, F32, U, a_weight, rows, weight64

pytestmark = pytest.mark.gpu


def check(out, x, w):
    m = weight64(w)
    ts = 1.0 if w.ts is None else w.ts.double().item()
    x = x.double()
    T, K = x.shape
    block = 32 if w.ts is None else 16
    y, size = (x @ m.T) * ts, (x.abs() @ m.abs().T) * abs(ts)
    most = x.abs().view(T, -1, block).amax(2)
    off = most * 2.0 ** -22
    if w.ts is not None:
        off = torch.maximum(off, most.amax(1, keepdim=True) * 2.0 ** -30)
    off = off.repeat_interleave(block, 1) @ m.abs().T * abs(ts)
    half = torch.finfo(out.dtype).eps / 2
    least = torch.finfo(out.dtype).smallest_normal * half
    tol = (K / 4 + 20) * U * size + off
    assert ((out.double() - y).abs() <= tol * (1 + half) + y.abs() * half + least).all()


def enough(T, K, more, fmt="nvfp4"):
    """The fewest rows that make a product of T tokens one for this path, and some."""
    least = 1 << 28 if T <= 8 else 1 << 25 if T <= 16 else -(-(1 << 24) // -(-T // 32))
    N = -(-least // K)
    size = moe.lib().moe_linear_fp4_workspace
    code = moe.WEIGHTS_NVFP4 if fmt == "nvfp4" else moe.WEIGHTS_MXFP4
    assert size(code, T, N, K) > 0 and size(code, T, N - 1, K) == 0
    return N + more


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,more,K", [(1, 1, 8192), (3, 255, 4096), (7, 0, 16384), (9, 1, 512), (10, 129, 1024), (12, 256, 4096), (15, 300, 8192),
                                      (16, 6, 32768), (16, 7, 65536), (17, 257, 1024), (20, 900, 512), (24, 3, 3584), (48, 140, 8192), (64, 2, 65536),
                                      (255, 70, 512), (257, 40, 1024), (261, 600, 512), (530, 33, 512)])
def test_against_64_bits(T, more, K, dt, fmt):
    N = enough(T, K, more, fmt)
    x, w = rows(T, K, dt, T + K), a_weight(N, K, fmt, N + K)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i in range(0, N, 1 << 14):                                # the weight in 64 bits, a piece at a time
        check(out[:, i:i + (1 << 14)], x, moe.NvfpTensor(w.codes[i:i + (1 << 14)], w.scales[i:i + (1 << 14)], w.ts))
    assert torch.equal(moe.linear_fp4(x, w), out.to(dt))
    assert torch.equal(moe.linear_fp4(x, w, out_dtype=F32), out)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("step", [1, 5, 9, 12, 20, 40])
def test_blocks_of_any_size_beside_one_another(step, fmt):
    """Scale blocks 2^-step times the one before: a block's integers reach far below the token's largest value and not."""
    K, T = 8192, 19
    block = 16 if fmt == "nvfp4" else 32
    x = rows(T, K, F32, step)
    x = (x.view(T, -1, block) * 2.0 ** (-step * (torch.arange(K // block, device="cuda") % 4)).view(1, -1, 1)).reshape(T, K).to(BF)
    w = a_weight(enough(T, K, 1, fmt), K, fmt, step)
    check(moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("exponent", [-120, -60, 0, 60, 112])
def test_rows_of_any_size(exponent):
    K, T = 8192, 20
    N = enough(T, K, 0)
    w = moe.NvfpTensor(a_weight(N, K, "nvfp4").codes, torch.full((N, K // 16), 0x08, dtype=torch.uint8, device="cuda"),
                       torch.tensor([1.0], device="cuda"))
    x = (rows(T, K, F32, 7).double() * 2.0 ** exponent).to(BF)
    x[1] = 0
    x[2, ::2] = 2.0 ** -126
    x[4] = 2.0 ** -130
    out = moe.linear_fp4(x, w, out_dtype=F32)
    check(out, x, w)
    assert (out[1] == 0).all()


def test_mxfp4_scales_of_any_size():
    K, T = 8192, 18
    N = enough(T, K, 48, "mxfp4")
    w = a_weight(N, K, "mxfp4")
    w.scales[:16] = 30
    w.scales[16:32] = 215
    w.scales[32:, ::2], w.scales[32:, 1::2] = 40, 200
    x = rows(T, K, BF, 9)
    check(moe.linear_fp4(x, w, out_dtype=F32), x, w)
    only = x.clone()
    only.view(T, K // 64, 2, 32)[:, :, 1] = 0
    check(moe.linear_fp4(only, w, out_dtype=F32), only, w)
    w.scales[7, 3] = 255
    bad = moe.linear_fp4(x, w, out_dtype=F32)
    assert bad[:, 7].isnan().all() and bad.isnan().sum() == T


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", [512, 8192])
def test_infinities_and_nans_stay_in_their_rows(K, fmt):
    w, x = a_weight(enough(20, K, 9, fmt), K, fmt), rows(20, K, BF)
    fine = moe.linear_fp4(x, w, out_dtype=F32)
    x[3] = float("nan")
    x[5, 17] = float("inf")
    x[18, K - 1] = -float("inf")
    x[19, 40], x[19, K - 3] = float("inf"), float("inf")
    bad = moe.linear_fp4(x, w, out_dtype=F32)
    keep = [i for i in range(20) if i not in (3, 5, 18, 19)]
    assert torch.equal(bad[keep], fine[keep]) and bad[3].isnan().all()
    m = weight64(w)
    for row in (5, 18, 19):
        want = (x[row].double()[None] * m).sum(1)
        assert torch.equal(bad[row].isnan(), want.isnan())
        there = ~want.isnan()
        assert torch.equal(bad[row][there], want[there].float())


def test_scales_that_are_nan_or_zero_stay_in_their_rows():
    T, K = 20, 1024
    N = enough(T, K, 5)
    w, x = a_weight(N, K, "nvfp4"), rows(T, K, BF, 6)
    fine = moe.linear_fp4(x, w, out_dtype=F32)
    w.scales[130, 3], w.scales[N - 1, 0] = 0x7F, 0x7F             # E4M3's NaN
    w.scales[7] = 0
    out = moe.linear_fp4(x, w, out_dtype=F32)
    assert out[:, 130].isnan().all() and out[:, N - 1].isnan().all() and (out[:, 7] == 0).all()
    keep = [i for i in range(N) if i not in (7, 130, N - 1)]
    assert torch.equal(out[:, keep], fine[:, keep])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_a_token_does_not_depend_on_the_others(fmt):
    w, x = a_weight(enough(9, 1024, 200, fmt), 1024, fmt), rows(32, 1024, BF)
    every = moe.linear_fp4(x[:16], w, out_dtype=F32)
    for T in (9, 11, 15):
        assert torch.equal(moe.linear_fp4(x[:T], w, out_dtype=F32), every[:T])
    assert torch.equal(moe.linear_fp4(x, w, out_dtype=F32)[:16], every)


def test_strided_rows():
    T, K = 21, 768
    w = a_weight(enough(T, K, 70), K, "nvfp4")
    for dt in (BF, F16):
        x = torch.full((T, 1000), float("nan"), dtype=dt, device="cuda")[:, 8:8 + K]
        x.copy_(rows(T, K, dt, 4))
        assert torch.equal(moe.linear_fp4(x, w), moe.linear_fp4(x.contiguous(), w))
        check(moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("K,N", [(2048, 9000), (16384, 1100)])
def test_weights_written_by_the_call_before_and_graphs_and_streams(K, N):
    """The product's blocks load weights early: never before the calls in front have written them."""
    T = 24
    assert moe.lib().moe_linear_fp4_workspace(moe.WEIGHTS_NVFP4, T, N, K) > 0
    x, w32 = rows(T, K, BF, 11), 0.02 * torch.randn(N, K, device="cuda")
    w = moe.quantize_nvfp4(w32)
    moe.linear_fp4(x, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.quantize_nvfp4(w32, out=w)
        one = moe.linear_fp4(x, w)
        two = moe.linear_fp4(x * 2, w)
    side = torch.cuda.Stream()
    for seed in (12, 13, 14):
        x.copy_(rows(T, K, BF, seed))
        w32.copy_(0.02 * torch.randn(N, K, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        check(one, x, w)
        assert torch.equal(two, one * 2)
        got = [moe.linear_fp4(x, w, stream=side), moe.linear_fp4(x, w)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], one) and torch.equal(got[1], one)
    for seed in range(20, 30):                                    # each call with the weight changed just before
        w32.copy_(0.02 * torch.randn(N, K, device="cuda"))
        moe.quantize_nvfp4(w32, out=w)
        check(moe.linear_fp4(x, w, out_dtype=F32), x, w)


def test_two_calls_behind_one_another_share_nothing():
    """The second reads what the first writes; both have workspaces, given back at once."""
    K = N = 4096
    T = 40
    a, b = a_weight(N, K, "nvfp4", 1), a_weight(N, K, "mxfp4", 2)
    a.ts.fill_(1e-4)
    x = rows(T, K, BF, 3)
    for _ in range(5):
        y = moe.linear_fp4(x, a)
        z = moe.linear_fp4(y, b, out_dtype=F32)
        check(z, y, b)
        check(y, x, a)
