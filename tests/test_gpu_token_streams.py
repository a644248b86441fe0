"""Token path calls on a stream of the caller's: inputs freed right behind the call keep their values until it has run."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu


def test_inputs_freed_behind_a_call_on_another_stream():
    T, H, k, E = 512, 1024, 4, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    bf = torch.bfloat16
    w = torch.ones(H, device="cuda", dtype=bf)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    order = moe.sort_pairs(ids, E, align=8)
    R = order["sorted_rows"].shape[0]
    p = torch.rand(T, k, generator=g, device="cuda")
    kept = {n: torch.randn(shape, generator=g, device="cuda").to(bf) for n, shape in
            dict(x=(T, H), r=(T, H), rows=(R, H), go=(T, H)).items()}
    rstd = moe.rms_norm(kept["x"], w)["rstd"]
    side = torch.cuda.Stream()

    def calls(t, stream):
        return [moe.rms_norm(t["x"], w, residual=t["r"], stream=stream)["y"],
                moe.rms_norm_backward(t["go"], t["x"], w, rstd, grad_sum=t["r"], stream=stream)["grad_sum"],
                moe.dispatch(t["x"], order, stream=stream)["rows"],
                moe.combine(t["rows"], order, p, base=t["r"], stream=stream),
                moe.dispatch_backward(t["rows"], order, stream=stream),
                moe.combine_backward(t["go"], t["rows"], order, p, stream=stream)["grad_y"]]

    want = calls(kept, None)
    torch.cuda.synchronize()
    for i in range(len(want)):
        gone = {n: v.clone() for n, v in kept.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                # some 10 ms: the call waits behind it
        got = calls(gone, side)[i]
        gone.clear()                                     # freed while the call has yet to run
        again = [torch.full(v.shape, 7.0, device="cuda", dtype=bf) for v in kept.values() for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want[i]), i
        del again
