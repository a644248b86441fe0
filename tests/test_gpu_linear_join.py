"""linear_fp4 on the tensor cores where a cluster's blocks join the parts of several items one behind the other."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_linear import BF, F32, a_weight, rows
from test_gpu_linear_tokens import check

pytestmark = pytest.mark.gpu


# four parts in five and three rounds, eight parts in three
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(20, 20480, 16384), (12, 24500, 16384), (12, 10000, 65536)])
def test_parts_of_several_items(T, N, K, fmt):
    w = a_weight(N, K, fmt, 5)
    xs = [rows(T, K, BF, i) for i in range(3)]
    first = [moe.linear_fp4(x, w, out_dtype=F32) for x in xs]
    for x, out in zip(xs, first):
        for i in range(0, N, 1 << 12):
            check(out[:, i:i + (1 << 12)], x, moe.NvfpTensor(w.codes[i:i + (1 << 12)], w.scales[i:i + (1 << 12)], w.ts))
    again = [moe.linear_fp4(xs[i % 3], w, out_dtype=F32) for i in range(60)]        # nothing waits between
    for i, out in enumerate(again):
        assert torch.equal(out, first[i % 3])
