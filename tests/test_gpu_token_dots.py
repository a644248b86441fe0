"""combine_backward's dot products against 64 bits, within what the additions of the split taken can round.

With u = 2^-24: a thread's sum of a piece's values is a chain of half as many multiply-adds and one addition (the other
half's chain is no longer), then 5 levels over a warp and, where a block takes a row, a chain over its warps."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def roundings(T, k, H, dtype):
    values = 16 // dtype.itemsize                        # of a 16-byte piece
    pieces = H // values
    few = T <= 152
    batch = 2 if few or k <= 2 else 4 if k <= 4 else 5 if k in (5, 9, 10) else 8
    if not few and pieces <= 32 * (4 if batch > 4 else 8):
        threads, warps = 32, 1                           # a token a warp
    else:
        at_once = 2 if batch == 5 else 8 // batch
        threads = max(128 if few else 32, min(256, -(-(-(-pieces // at_once)) // 32) * 32))
        warps = threads // 32
    return -(-pieces // threads) * (values // 2 + 1) + 5 + warps


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(3, 8, 4096), (152, 3, 16384), (153, 2, 2048), (153, 2, 2056), (400, 4, 1840), (400, 3, 8192),
                                   (400, 8, 512), (400, 8, 1024), (400, 8, 1032), (400, 7, 65536), (160, 5, 1024), (160, 9, 16384)])
def test_dot_products(T, k, H, dtype):
    E = 32
    g = torch.Generator(device="cuda").manual_seed(T + H)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    order = moe.sort_pairs(ids, E, align=8)
    # values of one sign: every partial sum is as large as it can be, and so is its rounding
    y = (1 + torch.rand(order["sorted_rows"].shape[0], H, generator=g, device="cuda")).to(dtype)
    go = (1 + torch.rand(T, H, generator=g, device="cuda")).to(dtype)
    got = moe.combine_backward(go, y, order, torch.rand(T, k, generator=g, device="cuda"))["grad_w"].double()
    inv = order["pair_rows"].long()
    for j in range(k):
        want = (go.double() * y[inv[:, j]].double()).sum(1)
        assert ((got[:, j] - want).abs() <= roundings(T, k, H, dtype) * U * want).all()
