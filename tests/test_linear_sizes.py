"""The size rule of linear_fp4 as the binding has it: a product of fewer than 2^28 multiplications is never asked for a
workspace (no GPU needed)."""
import pytest

import moe_routed_expert_router_gb300 as moe


@pytest.mark.parametrize("fmt,step", [(moe.WEIGHTS_NVFP4, 256), (moe.WEIGHTS_MXFP4, 512)])
@pytest.mark.parametrize("T", [*range(1, 70), 96, 97, 128, 255, 256, 257, 1000, 4096, 65536, 1 << 20])
def test_what_the_binding_does_not_ask_for_is_never_wanted(T, fmt, step):
    """The fewest rows for which the library wants a workspace, at every K: no fewer than the binding asks from."""
    size = moe.lib().moe_linear_fp4_workspace
    for K in range(step, 65537, step * (1 if T < 40 else 7)):
        most = ((1 << 28) - 1) // (T * K)                         # rows of the largest product that the binding does not ask for
        if most >= 1:
            assert size(fmt, T, most, K) == 0 and (T * most * K) >> 28 == 0
        assert size(fmt, T, (1 << 31) - 1025, K) > 0


def test_rows_of_f16_want_more_work():
    """Each type's rule, and that the size for any type is the larger."""
    any_type, size = moe.lib().moe_linear_fp4_workspace, moe.lib().moe_linear_fp4_workspace_for
    nv, mx, bf, f16 = moe.WEIGHTS_NVFP4, moe.WEIGHTS_MXFP4, moe.DTYPE_BF16, moe.DTYPE_F16
    for fmt, dt, T, least in ((nv, bf, 8, 1 << 28), (nv, f16, 8, 1 << 28), (mx, bf, 1, 1 << 28), (mx, f16, 1, 3 << 27), (nv, bf, 9, 1 << 25),
                              (mx, f16, 16, 3 << 25), (nv, bf, 32, 1 << 24), (nv, f16, 17, 5 << 23), (mx, f16, 64, 5 << 22), (mx, bf, 64, 1 << 23)):
        K = 512
        N = -(-least // K)
        assert size(fmt, dt, T, N, K) > 0 and size(fmt, dt, T, N - 1, K) == 0
    for fmt in (nv, mx):
        for T in (1, 8, 9, 16, 17, 32, 33, 64, 300):
            for N in (1000, 8192, 16400, 65536, 200000, 800000):
                for K in (512, 2048, 4096):
                    sizes = [size(fmt, dt, T, N, K) for dt in (bf, f16)]
                    assert any_type(fmt, T, N, K) == max(sizes) and size(fmt, moe.DTYPE_F32, T, N, K) == 0


def test_a_product_without_a_workspace_is_refused_by_its_own_types_rule():
    import ctypes
    w = moe.Nvfp4(256, 256, 256)
    L = moe.lib()

    def call(dt, x):
        return L.moe_linear_fp4(x, 512, ctypes.byref(w), moe.WEIGHTS_NVFP4, 16, 1 << 17, 512, dt, dt, 256, None, 0, None)
    assert L.moe_linear_fp4_workspace_for(moe.WEIGHTS_NVFP4, moe.DTYPE_BF16, 16, 1 << 17, 512) > 0
    assert L.moe_linear_fp4_workspace_for(moe.WEIGHTS_NVFP4, moe.DTYPE_F16, 16, 1 << 17, 512) == 0
    assert call(moe.DTYPE_BF16, 256 + 8) == moe.ERR_INVALID_ARG   # the workspace first
    assert call(moe.DTYPE_F16, 256 + 8) == moe.ERR_MISALIGNED     # it needs none: refused for x
