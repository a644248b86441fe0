"""The workspace of rms_norm's backward pass by element type (no GPU needed: every call is refused)."""
import pytest

import moe_routed_expert_router_gb300 as moe

A = 256                       # an aligned address that is never used
TYPES = [moe.DTYPE_F32, moe.DTYPE_BF16, moe.DTYPE_F16]


def back(T, H, dt, ws, n):
    """Refused in every case: for its workspace, or after that for a misaligned grad_sum."""
    return moe.lib().moe_rms_norm_backward(A, A, A, A, A + 8, T, H, dt, A, A, ws, n, None)


@pytest.mark.parametrize("T,H", [(3, 520), (8, 1000), (16, 1024)])
def test_16_bit_rows_that_one_block_takes_need_none(T, H):
    """Rows of 513 to 1024 values take a warp each in 16 bits and a block each in fp32."""
    size = moe.lib().moe_rms_norm_backward_workspace_for
    assert size(T, H, moe.DTYPE_BF16) == size(T, H, moe.DTYPE_F16) == 0 and size(T, H, moe.DTYPE_F32) == 4 * T * H
    for dt in TYPES[1:]:
        assert back(T, H, dt, None, 0) == moe.ERR_MISALIGNED
    assert back(T, H, moe.DTYPE_F32, None, 0) == moe.ERR_INVALID_ARG


@pytest.mark.parametrize("T,H", [(1, 8), (2, 4096), (17, 264), (300, 512), (400, 520), (5000, 1024), (5000, 1032), (9000, 4528), (1 << 30, 16384)])
def test_what_is_asked_for_is_what_is_checked(T, H):
    L = moe.lib()
    sizes = [L.moe_rms_norm_backward_workspace_for(T, H, dt) for dt in TYPES]
    assert L.moe_rms_norm_backward_workspace(T, H) == max(sizes)      # enough for any type
    for dt, n in zip(TYPES, sizes):
        assert back(T, H, dt, A if n else None, n) == moe.ERR_MISALIGNED
        if n:
            assert back(T, H, dt, A, n - 1) == moe.ERR_INVALID_ARG and back(T, H, dt, None, n) == moe.ERR_INVALID_ARG


def test_sizes_that_the_call_refuses_need_none():
    size = moe.lib().moe_rms_norm_backward_workspace_for
    assert size(0, 256, 1) == size(-1, 256, 1) == size(400, 0, 1) == size(400, 256, 3) == size(400, 256, -1) == 0
