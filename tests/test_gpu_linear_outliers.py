"""linear_fp4 on the block-scaled tensor cores: a row with one channel far above the others, whose weights are zero, keeps
what the other channels give.  A value is off by half a step of its scale block's integers, 2^-22 of the block's largest
value, or for NVFP4 2^-39 of the token's where that is more; the sums as in test_gpu_linear."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_linear import BF, F16, F32, U, a_weight, rows, weight64
from test_gpu_linear_tokens import enough

pytestmark = pytest.mark.gpu


def check(out, x, w):
    m, ts, x = weight64(w), w.ts.double().item(), x.double()
    T, K = x.shape
    y, size = (x @ m.T) * ts, (x.abs() @ m.abs().T) * ts
    most = x.abs().view(T, -1, 16).amax(2)
    off = torch.maximum(most * 2.0 ** -22, most.amax(1, keepdim=True) * 2.0 ** -39).repeat_interleave(16, 1) @ m.abs().T * ts
    assert ((out.double() - y).abs() <= ((K / 4 + 20) * U * size + off) * (1 + U) + y.abs() * U + 2.0 ** -149).all()


@pytest.mark.parametrize("times", [10, 14, 18, 22, 26, 30, 36, 45])
@pytest.mark.parametrize("T,K", [(20, 1024), (16, 2048), (3, 8192)])
def test_an_outlier_channel_without_weights(T, K, times):
    """bf16 rows: the whole scale block of the outlier has codes of zero, so nothing of it is in the sum."""
    w = a_weight(enough(T, K, 3), K, "nvfp4", times)
    w.codes[:, 64:72] = 0                                         # values 128 to 143
    x = rows(T, K, BF, times)
    x[:, 133] = 2.0 ** times
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i in range(0, out.shape[1], 1 << 13):
        check(out[:, i:i + (1 << 13)], x, moe.NvfpTensor(w.codes[i:i + (1 << 13)], w.scales[i:i + (1 << 13)], w.ts))


@pytest.mark.parametrize("times", [14, 20, 24])
def test_an_outlier_channel_of_f16_rows(times):
    T, K = 20, 1024
    w = a_weight(enough(T, K, 3), K, "nvfp4", times)
    w.codes[:, 64:72] = 0
    x = (rows(T, K, F32, times) * 2.0 ** -10).to(F16)
    x[:, 133] = 2.0 ** (times - 10)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    for i in range(0, out.shape[1], 1 << 13):
        check(out[:, i:i + (1 << 13)], x, moe.NvfpTensor(w.codes[i:i + (1 << 13)], w.scales[i:i + (1 << 13)], w.ts))
