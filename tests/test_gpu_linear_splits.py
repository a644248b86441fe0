"""linear_fp4 where the warps' rings and sums take nearly all of a block's shared memory: splits into 11 warps, with many
tiles and several passes.  The tolerance is test_gpu_linear's."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_linear import BF, F16, F32, a_weight, check, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,N,K", [(1, 25600, 2816), (8, 24321, 2688), (9, 30000, 2688), (16, 18000, 2688), (16, 19456, 2816), (32, 18000, 1408),
                                   (32, 17025, 1408), (64, 9000, 1408), (64, 28000, 1408)])
def test_splits_that_fill_the_shared_memory(T, N, K, dt, fmt):
    x, w = rows(T, K, dt, T + K), a_weight(N, K, fmt, N + K)
    out = moe.linear_fp4(x, w, out_dtype=F32)
    check(out, x, w)
    assert torch.equal(moe.linear_fp4(x, w), out.to(dt))


def test_weights_past_four_gigabytes():
    """Code offsets beyond 32 bits: the last rows of a weight of 4.5 GB whose K keeps it on the warp kernel."""
    K = 65536 - 128
    N = (1 << 32) // (K // 2) + 5000
    assert moe.lib().moe_linear_fp4_workspace(moe.WEIGHTS_NVFP4, 3, N, K) == 0
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda")          # 1
    tail = a_weight(300, K, "nvfp4")
    codes[-300:], scales[-300:] = tail.codes, tail.scales
    ts = torch.tensor([0.0173], device="cuda")
    x = rows(3, K, F16, 5)
    out = moe.linear_fp4(x, moe.NvfpTensor(codes, scales, ts), out_dtype=F32)
    assert (out[:, :-300] == 0).all()
    check(out[:, -300:], x, moe.NvfpTensor(tail.codes, tail.scales, ts))
