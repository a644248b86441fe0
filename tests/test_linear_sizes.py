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
