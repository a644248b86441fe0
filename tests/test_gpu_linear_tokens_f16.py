"""linear_fp4 of f16 rows at the sizes that take them to the block-scaled tensor cores, and just below."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
import test_gpu_linear_outliers as outliers
from test_gpu_linear import F16, F32, a_weight, rows, weight64
from test_gpu_linear_tokens import check

pytestmark = pytest.mark.gpu


def least_rows(T, K, fmt):
    least = (3 << 27 if fmt == "mxfp4" else 1 << 28) if T <= 8 else 3 << 25 if T <= 16 else -(-(5 << 23) // -(-T // 32))
    N = -(-least // K)
    size = moe.lib().moe_linear_fp4_workspace_for
    code = moe.WEIGHTS_NVFP4 if fmt == "nvfp4" else moe.WEIGHTS_MXFP4
    assert size(code, moe.DTYPE_F16, T, N, K) > 0 and size(code, moe.DTYPE_F16, T, N - 1, K) == 0
    return N


def pieces(w, n=1 << 13):
    return [(i, moe.NvfpTensor(w.codes[i:i + n], w.scales[i:i + n], w.ts)) for i in range(0, w.codes.shape[0], n)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,more,K", [(1, 1, 8192), (5, 255, 16384), (9, 1, 512), (12, 256, 4096), (16, 7, 65536), (17, 257, 1024), (24, 3, 3584), (64, 2, 65536),
                                      (257, 40, 1024), (530, 33, 512), (8, -1, 8192), (16, -1, 4096), (17, -1, 1024), (64, -1, 2048)])
def test_against_64_bits(T, more, K, fmt):
    N = least_rows(T, K, fmt) + more
    x, w = rows(T, K, F16, T + K), a_weight(N, K, fmt, N + K)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i, part in pieces(w):
        check(out[:, i:i + (1 << 13)], x, part)
    assert torch.equal(moe.linear_fp4(x, w), out.to(F16))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_strided_rows_with_infinities_and_nans(fmt):
    T, K = 21, 1024
    w = a_weight(least_rows(T, K, fmt) + 70, K, fmt)
    x = torch.full((T, 1200), float("nan"), dtype=F16, device="cuda")[:, 8:8 + K]
    x.copy_(rows(T, K, F16, 4))
    fine = moe.linear_fp4(x, w, out_dtype=F32)
    assert torch.equal(fine, moe.linear_fp4(x.contiguous(), w, out_dtype=F32))
    for i, part in pieces(w):
        check(fine[:, i:i + (1 << 13)], x, part)
    x[3], x[5, 17], x[20, K - 1] = float("nan"), float("inf"), -float("inf")
    bad = moe.linear_fp4(x, w, out_dtype=F32)
    keep = [i for i in range(T) if i not in (3, 5, 20)]
    assert torch.equal(bad[keep], fine[keep]) and bad[3].isnan().all()
    m = weight64(w)
    for row in (5, 20):
        want = (x[row].double()[None] * m).sum(1)
        assert torch.equal(bad[row].isnan(), want.isnan())
        there = ~want.isnan()
        assert torch.equal(bad[row][there], want[there].float())


def test_f16_rows_below_the_rule_keep_every_bit():
    """Between the types' borders f16 rows enter as they are: an outlier takes nothing from the values beside it."""
    T, N, K = 20, 40000, 512
    assert moe.lib().moe_linear_fp4_workspace_for(moe.WEIGHTS_NVFP4, moe.DTYPE_BF16, T, N, K) > 0
    assert moe.lib().moe_linear_fp4_workspace_for(moe.WEIGHTS_NVFP4, moe.DTYPE_F16, T, N, K) == 0
    w = a_weight(N, K, "nvfp4")
    w.codes[:, 66] = 0                                            # values 132 and 133
    x = (rows(T, K, torch.float32, 3) * 2.0 ** -12).to(F16)
    base = moe.linear_fp4(x, w, out_dtype=F32)
    y = x.clone()
    y[:, 133] = 60000.0
    assert torch.equal(moe.linear_fp4(y, w, out_dtype=F32), base)


@pytest.mark.parametrize("exponent,byte", [(0, 238), (-12, 250), (6, 0)])
def test_mxfp4_scales_to_their_ends(exponent, byte):
    T, K = 20, 512
    w = a_weight(least_rows(T, K, "mxfp4") + 1, K, "mxfp4", byte)
    w.scales.fill_(byte)
    x = (rows(T, K, F32, 8) * 2.0 ** exponent).to(F16)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    assert out.isfinite().all()
    for i, part in pieces(w):
        check(out[:, i:i + (1 << 13)], x, part)


@pytest.mark.parametrize("times", [14, 20, 24])
def test_an_outlier_channel_without_weights(times):
    T, K = 20, 1024
    w = a_weight(least_rows(T, K, "nvfp4") + 3, K, "nvfp4", times)
    w.codes[:, 64:72] = 0                                         # values 128 to 143
    x = (rows(T, K, F32, times) * 2.0 ** -10).to(F16)
    x[:, 133] = 2.0 ** (times - 10)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i, part in pieces(w):
        outliers.check(out[:, i:i + (1 << 13)], x, part)
