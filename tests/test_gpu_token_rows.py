"""The largest number of tokens that the token path takes, 2^31 - 1, with rows of 16 bytes."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

T, H = (1 << 31) - 1, 8
BF = torch.bfloat16
SOME = [0, 1, 7, 8, 1 << 29, (1 << 30) + 3, T - 9, T - 8, T - 7, T - 2, T - 1]


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _all(rows, value):
    """Whether every value of rows is that one, a piece at a time."""
    return all((piece == value).all().item() for piece in rows.split(1 << 28))


def _order():
    """Eight expert rows, held by tokens of SOME."""
    inv = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    rows = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    for r, t in enumerate(SOME[-8:]):
        inv[t, 0], rows[r] = r, t
    return dict(sorted_rows=rows, pair_rows=inv)


def test_norm(room):
    x = torch.full((T, H), 2.0, dtype=BF, device="cuda")
    for t in SOME:
        x[t, ::2] = 0
    out = dict(y=torch.full((T, H), float("nan"), dtype=BF, device="cuda"))
    moe.rms_norm(x, torch.ones(H, dtype=BF, device="cuda"), out=out)
    for t in SOME:                                       # half of the values are zero: 2 / sqrt(2)
        want = torch.tensor([0, 2 ** 0.5], device="cuda").repeat(4).to(BF)
        assert torch.equal(out["y"][t], want), t
        out["y"][t] = 1
    assert _all(out["y"], 1)


def test_dispatch(room):
    order = _order()
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    for t in SOME:
        x[t] = t % 251
    rows = moe.dispatch(x, order)["rows"]
    assert torch.equal(rows, x[torch.tensor(SOME[-8:], device="cuda")])


def test_combine_and_its_gradients(room):
    order = _order()
    y = torch.arange(1, 9, device="cuda").to(BF)[:, None].repeat(1, H)
    out = torch.full((T, H), float("nan"), dtype=BF, device="cuda")
    moe.combine(y, order, out=out)
    for r, t in enumerate(SOME[-8:]):
        assert (out[t] == r + 1).all()
        out[t] = 0
    assert _all(out, 0)
    for r, t in enumerate(SOME[-8:]):
        out[t] = r - 3                                   # the gradient that comes back
    w = torch.full((T, 1), 2.0, device="cuda")
    got = moe.combine_backward(out, y, order, w)
    for r, t in enumerate(SOME[-8:]):
        assert (got["grad_y"][r] == 2 * (r - 3)).all() and got["grad_w"][t, 0] == H * (r + 1) * (r - 3)
        got["grad_w"][t, 0] = 0
    assert _all(got["grad_w"], 0)
