"""rms_norm's 8-bit output where a group's products s * weight are tiny beside its norm.

With a small eps 1 / rms reaches 2^20 and more, so products below 448 / (largest fp32) = 2^-119.2 have norms above
the scale's bound of 2^-100; 448 over such a product is no fp32 number."""
import numpy as np
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_gpu_norm import N_REL, _check_quant

pytestmark = pytest.mark.gpu

# few rows; then rows enough for a warp a row, and for two and four pieces a thread
SHAPES = [(6, 512), (3, 4104), (5, 9216), (320, 264), (2100, 1000), (330, 2048), (400, 4104)]


@pytest.mark.parametrize("eps", [1e-12, 1e-16, 1e-20, 1e-30])
@pytest.mark.parametrize("quant", [moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW, moe.QUANT_MXFP8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_groups_of_tiny_products_and_zeros(T, H, dtype, quant, eps):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    G = {moe.QUANT_E4M3_128: 128, moe.QUANT_MXFP8: 32}.get(quant, H)
    n_groups = -(-H // G)
    # a group's largest magnitude: 2^-119 down to the smallest normal number, and a few groups far above and below
    size = 2.0 ** -(119 + 7 * torch.rand(T, n_groups, generator=g, device="cuda", dtype=torch.float64))
    size = torch.where(torch.rand(T, n_groups, generator=g, device="cuda") < 0.2, size * 2.0 ** 30, size)
    size = torch.where(torch.rand(T, n_groups, generator=g, device="cuda") < 0.2, size * 2.0 ** -6, size)
    x = 2 * torch.rand(T, n_groups, G, generator=g, device="cuda", dtype=torch.float64) - 1
    x[torch.rand(T, n_groups, G, generator=g, device="cuda") < 0.3] = 0
    x = (x * size[:, :, None]).reshape(T, -1)[:, :H].contiguous().to(dtype)
    w = torch.ones(H, dtype=dtype, device="cuda")           # a product is the value itself: none of its bits is lost
    out = moe.rms_norm(x, w, eps=eps, quant=quant)
    s = x.double()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(np.float32(eps)))
    # squares below 2^-126 lose bits: up to half of 2^-149 each, against a sum of at least H * eps
    rel = N_REL + 2.0 ** -150 / float(np.float32(eps))
    codes = out["q"].float()
    assert codes.isfinite().all() and (codes[x == 0] == 0).all()
    _check_quant(n.cpu().numpy(), out["q"], out["scales"], quant, rel)


@pytest.mark.parametrize("quant", [moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW])
def test_one_value_and_zeros(quant):
    """The formula by hand: a group of one magnitude and zeros has codes 448 and 0."""
    x = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    x[0, ::2] = 1e-36
    out = moe.rms_norm(x, torch.ones(128, dtype=torch.bfloat16, device="cuda"), eps=1e-12, quant=quant)
    assert (out["q"][0, ::2].float() == 448).all() and (out["q"][0, 1::2].float() == 0).all()
    assert abs(out["scales"].item() * 448 / (x[0, 0].item() * 1e6) - 1) < 2.0 ** -20


@pytest.mark.parametrize("quant", [moe.QUANT_E4M3_128, moe.QUANT_E4M3_ROW])
def test_a_nan_weight_makes_its_group_nan(quant):
    x = torch.ones(2, 512, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    w[200] = float("nan")
    out = moe.rms_norm(x, w, quant=quant)
    assert out["scales"].isnan().any()
    values = out["q"].float() * (out["scales"].repeat_interleave(128, 1) if quant == moe.QUANT_E4M3_128 else out["scales"])
    group = slice(128, 256) if quant == moe.QUANT_E4M3_128 else slice(0, 512)
    assert values[:, group].isnan().all()
    if quant == moe.QUANT_E4M3_128:
        assert values[:, :128].isfinite().all() and values[:, 256:].isfinite().all()
