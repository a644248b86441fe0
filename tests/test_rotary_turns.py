"""rotary_turns over every frequency that it takes (no GPU needed)."""
import math
from fractions import Fraction

import pytest

import moe_routed_expert_router_gb300 as moe


@pytest.mark.parametrize("f", [0.0, 1.0, -1.0, 5e-324, -1e-20, 0.7, -0.7, 6.5, -1e5, 1e17, 1e290, 1e300, -1.7e308])
def test_any_finite_frequency(f):
    """The fraction of a turn of f / (2 pi) as 64-bit floating point has it, rounded down to 2^-64."""
    got = moe.rotary_turns(16, frequencies=[f] * 8, device="cpu").tolist()
    want = math.floor(Fraction(f / (2 * math.pi)) * 2 ** 64) % 2 ** 64
    assert [t % 2 ** 64 for t in got] == [want] * 8


@pytest.mark.parametrize("dim,base", [(64, 1e-320), (512, 5e-324)])
def test_a_base_whose_frequencies_are_too_large_is_refused(dim, base):
    with pytest.raises(moe.MoeError):
        moe.rotary_turns(dim, base=base, device="cpu")
