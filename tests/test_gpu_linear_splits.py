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
