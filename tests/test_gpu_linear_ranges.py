"""linear_fp4 at the ends of the scales' and rows' ranges: what fp32 arithmetic gives a number for has one, of both
kernels.  Tolerances are those of their own tests: they hold for any finite sum."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
import test_gpu_linear as small
import test_gpu_linear_tokens as large
from test_gpu_linear import BF, F16, F32, a_weight, rows

pytestmark = pytest.mark.gpu

KERNELS = [(5, "small"), (12, "small"), (20, "small"), (20, "large"), (6, "large")]


def shape(T, kernel, fmt):
    """K = 512 and rows enough for the kernel (8192 values where few tokens want many)."""
    K = 8192 if T <= 8 and kernel == "large" else 512
    return (large.enough(T, K, 1, fmt) if kernel == "large" else 70), K


def check(kernel, out, x, w):
    assert out.isfinite().all()
    for i in range(0, out.shape[1], 1 << 13):
        (large if kernel == "large" else small).check(out[:, i:i + (1 << 13)], x, moe.NvfpTensor(w.codes[i:i + (1 << 13)], w.scales[i:i + (1 << 13)], w.ts))


# sizes of the rows, and the largest byte of the E8M0 scales: the sum of K products of at most 6 * 256 stays below 2^127
@pytest.mark.parametrize("exponent,byte", [(0, 238), (-20, 254), (-60, 254), (-118, 254), (40, 195), (100, 130), (100, 3), (115, 0)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_mxfp4_scales_to_their_ends(T, kernel, exponent, byte):
    N, K = shape(T, kernel, "mxfp4")
    byte = min(byte, 234 - exponent) if K == 8192 else byte
    w = a_weight(N, K, "mxfp4", byte)
    w.scales.copy_(torch.clamp(w.scales.int() - 156 + byte, min=0).to(torch.uint8))      # from 60 below it
    x = (rows(T, K, F32, 7).double() * 2.0 ** exponent).to(BF)
    check(kernel, moe.linear_fp4(x, w, out_dtype=F32), x, w)
    w.scales.fill_(byte)
    check(kernel, moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("exponent,byte", [(0, 238), (-12, 250), (6, 0)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_mxfp4_scales_to_their_ends_of_f16_rows(T, kernel, exponent, byte):
    N, K = shape(T, kernel, "mxfp4")
    byte = min(byte, 234 - exponent) if K == 8192 else byte
    w = a_weight(N, K, "mxfp4", byte)
    w.scales.fill_(byte)
    x = (rows(T, K, F32, 8) * 2.0 ** exponent).to(F16)
    check(kernel, moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("T,kernel", KERNELS)
def test_mxfp4_largest_scales_over_codes_of_zero(T, kernel):
    """Zeros times any finite scale are zeros, beside rows and values of any size."""
    N, K = shape(T, kernel, "mxfp4")
    w = a_weight(N, K, "mxfp4", 1)
    w.scales[:, 3::4] = 254
    w.codes.view(N, K // 32, 16)[:, 3::4] = 0
    x = rows(T, K, BF, 9)
    x.view(T, K // 32, 32)[:, 3::4] *= 2.0 ** 100
    x[1] *= 2.0 ** 20
    out = moe.linear_fp4(x, w, out_dtype=F32)
    assert out.isfinite().all()
    w.codes.view(N, K // 32, 16)[:, 3::4] = 0x88                  # negative ones
    assert torch.equal(moe.linear_fp4(x, w, out_dtype=F32), out)


# rows, tensor scale: a sum without the tensor scale passes fp32's largest number, or falls below its smallest normal one
@pytest.mark.parametrize("exponent,ts", [(117, 1.3e-7), (117, 2.0 ** -126), (112, -3e-9), (-116, 1.7e9), (-126, 2.0 ** 100), (0, 1e-45), (0, 0.0)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_nvfp4_tensor_scales_of_any_size(T, kernel, exponent, ts):
    N, K = shape(T, kernel, "nvfp4")
    w = a_weight(N, K, "nvfp4", 3)
    w.ts.fill_(ts)
    if exponent < 0:
        w.scales.fill_(0x08)                                      # 2^-6
    x = (rows(T, K, F32, 10).double() * 2.0 ** exponent).to(BF)
    check(kernel, moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("exponent,ts", [(-126, 2.0 ** 110), (-130, 1.1 * 2.0 ** 127), (-60, 2.0 ** 60), (118, -2.0 ** -149), (119, 2.0 ** -140), (-100, 2.0 ** -40)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_nvfp4_tensor_scales_over_the_least_and_largest_blocks(T, kernel, exponent, ts):
    """Scales of 2^-9 below rows that are small, of 448 above large ones, codes of every size."""
    N, K = shape(T, kernel, "nvfp4")
    w = a_weight(N, K, "nvfp4", 4)
    w.ts.fill_(ts)
    w.scales.fill_(0x01 if exponent < 0 else 0x7E)
    x = (torch.randn(T, K, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").double() * 2.0 ** exponent).to(BF)
    check(kernel, moe.linear_fp4(x, w, out_dtype=F32), x, w)


@pytest.mark.parametrize("exponent,ts", [(-109, 2.0 ** -20), (-118, 1.0), (-100, 1.7 * 2.0 ** -28)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_nvfp4_results_below_the_smallest_normal_number(T, kernel, exponent, ts):
    """There every operation on a sum rounds to half of 2^-149: two of a warp's stage, up to 4 stages a warp and 16 warps or 8
    parts joined, two of the tensor scale."""
    N, K = shape(T, kernel, "nvfp4")
    w = a_weight(N, K, "nvfp4", 4)
    w.ts.fill_(ts)
    w.scales.fill_(0x01)
    x = (torch.randn(T, K, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").double() * 2.0 ** exponent).to(BF)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i in range(0, N, 1 << 13):
        m = small.weight64(moe.NvfpTensor(w.codes[i:i + (1 << 13)], w.scales[i:i + (1 << 13)], w.ts))
        y = x.double() @ m.T * w.ts.double().item()
        size = x.double().abs() @ m.abs().T * abs(ts)
        off = 2.0 ** -22 * x.double().abs().amax(1, keepdim=True) * m.abs().sum(1) * abs(ts)
        assert ((out[:, i:i + (1 << 13)].double() - y).abs() <= 26 * 2.0 ** -150 + (K / 4 + 20) * small.U * size + off).all()
    assert (out != 0).any()
