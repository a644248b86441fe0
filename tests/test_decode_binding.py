"""What the binding of head_norm, linear_fp4 and decode_layer gives the library, without a GPU: stand-ins for the library,
for tensors on several devices and for the current device note what reaches the entry points."""
import pytest
import torch

import moe_routed_expert_router_gb300 as moe
from test_tokens_binding import Stream, Tensor, World

BF, F32, I32, U8, I64 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int64


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def every_call(index=0, stream=None, T=6, D=64, K=256, N=48, H=128, E=4, I=64, k=2, **change):
    """Each function on tensors of cuda:<index>: (name, call, the tensors it is given)."""
    def t(*shape, dtype=BF):
        return Tensor(shape, dtype, index)
    q, ke, qw, kw, pos, turns = t(T, 8, D), t(T, 2, D), t(D), t(D), t(T, dtype=I32), t(D // 2, dtype=I64)
    gq, gk = t(T, 8, D), t(T, 2, D)
    ho = dict(q=t(T, 8, D), k=t(T, 2, D))
    bo = dict(grad_q=t(T, 8, D), grad_k=t(T, 2, D), grad_qw=t(D, dtype=F32), grad_kw=t(D, dtype=F32))
    x, codes, scales, ts, lo = t(T, K), t(N, K // 2, dtype=U8), t(N, K // 16, dtype=U8), t(1, dtype=F32), t(T, N)
    rows, rw, bias, g, u, d, base = t(T, H), t(E, H, dtype=F32), t(E, dtype=F32), t(E, I, H), t(E, I, H), t(E, H, I), t(T, H)
    sh = (t(I, H), t(I, H), t(H, I))
    do = dict(out=t(T, H), topk_ids=t(T, k, dtype=I32), topk_w=t(T, k, dtype=F32))
    kw_ = dict(stream=stream)
    return [
        ("moe_head_norm", lambda: moe.head_norm(q, ke, qw, kw, pos, turns, out=ho, **kw_), [q, ke, qw, kw, pos, turns, *ho.values()]),
        ("moe_head_norm_backward", lambda: moe.head_norm_backward(gq, gk, q, ke, qw, kw, pos, turns, out=bo, **kw_),
         [q, ke, gq, gk, qw, kw, pos, turns, *bo.values()]),
        ("moe_linear_fp4", lambda: moe.linear_fp4(x, moe.NvfpTensor(codes, scales, ts), out=lo, **kw_), [x, codes, scales, ts, lo]),
        ("moe_decode_layer", lambda: moe.decode_layer(rows, rw, g, u, d, k, router_bias=bias, shared=sh, base=base, out=do, **kw_),
         [rows, rw, g, u, d, bias, base, *sh, *do.values()]),
    ]


def calls(world):
    return [c for c in world.calls if not c[0].endswith("_workspace")]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("given", [False, True])
def test_the_tensors_device_is_current_at_the_call(world, which, given):
    name, call, _ = every_call(1, Stream(1) if given else None)[which]
    call()
    (got, args, current), = calls(world)
    assert got == name and current == 1 and args[-1] == (7001 if given else 1001)
    assert world.current == 0
    world.current = 1
    before = world.switches
    call()
    assert world.switches == before and calls(world)[-1][2] == 1


@pytest.mark.parametrize("which", range(4))
def test_a_stream_of_another_device_is_refused(world, which):
    _, call, _ = every_call(0, Stream(1))[which]
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.ERR_INVALID_ARG and not calls(world)


@pytest.mark.parametrize("which", range(4))
def test_memory_of_the_tensors_is_held_for_a_given_stream(world, which):
    _, call, tensors = every_call(0)[which]
    call()
    assert not any(t.streams for t in tensors)
    stream = Stream(0)
    _, call, tensors = every_call(0, stream)[which]
    call()
    assert all(t.streams == [stream] for t in tensors)


@pytest.mark.parametrize("which,size", [(0, dict(T=1 << 31)), (0, dict(D=1 << 32)), (1, dict(T=(1 << 32) + 6)), (2, dict(T=1 << 31)),
                                        (2, dict(K=1 << 32)), (2, dict(N=(1 << 32) + 48)), (3, dict(T=1 << 31)), (3, dict(H=(1 << 32) + 128)),
                                        (3, dict(E=(1 << 32) + 4)), (3, dict(I=(1 << 32) + 64)), (3, dict(k=(1 << 32) + 2))])
def test_sizes_past_32_bits_are_refused(world, which, size):
    _, call, _ = every_call(**size)[which]
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.ERR_UNSUPPORTED_SHAPE and not calls(world)


@pytest.mark.parametrize("which,names", [(0, 4), (2, 1), (3, 10)])
def test_tensors_that_require_a_gradient_are_not_taken_in_silence(world, which, names):
    for i in range(names):
        name, call, tensors = every_call()[which]
        tensors[i].requires_grad = True
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.ERR_INVALID_ARG and "no_grad" in str(e.value) and not calls(world)
        with torch.no_grad():
            call()
        assert calls(world)[-1][0] == name
        world.calls.clear()


@pytest.mark.parametrize("which", range(4))
def test_every_tensor_has_to_be_on_the_device(world, which):
    """Each tensor on another device than the first, and each with one value more, is refused."""
    count = len(every_call()[which][2])
    for i in range(1, count):
        _, call, tensors = every_call()[which]
        tensors[i].index = 1
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.ERR_INVALID_ARG
        if i == 5 and which < 2 or i == 7 and which == 1:
            continue                                              # turns: another length is another rotation
        _, call, tensors = every_call()[which]
        t = tensors[i]
        t.meta = torch.empty((*t.meta.shape[:-1], t.meta.shape[-1] + 1), dtype=t.meta.dtype, device="meta")
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.ERR_INVALID_ARG
    assert not calls(world)


def test_arguments_in_their_places(world):
    T, D = 6, 64
    qkv = Tensor((T, 12, D), BF)
    q, k = Tensor((T, 8, D), BF), Tensor((T, 2, D), BF)
    q.meta, k.meta = qkv.meta[:, :8], qkv.meta[:, 8:10]           # parts of rows: tokens 12 heads apart
    w, pos, turns = Tensor((D,), BF), Tensor((T,), I32), Tensor((16,), I64)
    moe.head_norm(q, k, w, w, pos, turns, interleaved=True, eps=1e-5, out=dict(q=q, k=Tensor((T, 2, D), BF)))
    (_, a, _), = calls(world)
    assert a[1] == a[3] == 12 * D and a[8:16] == (T, 8, 2, D, 32, 1, moe.DTYPE_BF16, 1e-5) and a[17] == 12 * D and a[19] == 2 * D
    none = Tensor((0,), I64)
    moe.head_norm(q, k, w, w, pos, none, out=dict(q=q, k=k))      # no rotation: positions and turns are not given on
    assert calls(world)[-1][1][6:8] == (None, None) and calls(world)[-1][1][12] == 0
    odd = Tensor((T, 8, D), BF)
    odd.meta = torch.empty(T, 8, 2 * D, dtype=BF, device="meta")[:, :, :D]        # heads that are not behind one another
    with pytest.raises(moe.MoeError):
        moe.head_norm(odd, k, w, w, pos, turns)


def test_formats_and_types_of_a_4_bit_weight(world):
    x, out = Tensor((3, 256), torch.float16), Tensor((3, 40), F32)
    codes = Tensor((1, 40, 128), U8)
    moe.linear_fp4(x, moe.NvfpTensor(codes, Tensor((1, 40, 8), U8), None), out=out)
    a = calls(world)[-1][1]
    assert a[3:9] == (moe.WEIGHTS_MXFP4, 3, 40, 256, moe.DTYPE_F16, moe.DTYPE_F32)
    moe.linear_fp4(x, moe.NvfpTensor(codes, Tensor((1, 40, 16), U8), Tensor((), F32)), out=Tensor((3, 40), torch.float16))
    a = calls(world)[-1][1]
    assert a[3:9] == (moe.WEIGHTS_NVFP4, 3, 40, 256, moe.DTYPE_F16, moe.DTYPE_F16)
    n = len(calls(world))
    scales, ts = Tensor((1, 40, 16), U8), Tensor((1,), F32)
    for bad in (lambda: moe.linear_fp4(Tensor((3, 256), F32), moe.NvfpTensor(codes, scales, ts)),
                lambda: moe.linear_fp4(x, moe.NvfpTensor(Tensor((2, 40, 128), U8), Tensor((2, 40, 16), U8), ts)),
                lambda: moe.linear_fp4(x, moe.NvfpTensor(codes, scales, Tensor((2,), F32)), out=out),
                lambda: moe.linear_fp4(x, moe.NvfpTensor(codes, scales, ts), out=Tensor((3, 40), BF)),
                lambda: moe.linear_fp4(x, moe.NvfpTensor(codes, scales, ts), out=out, out_dtype=torch.float16)):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.status == moe.ERR_INVALID_ARG
    assert len(calls(world)) == n


@pytest.mark.parametrize("router", [2, -1, 1 << 32])
def test_routers_that_there_are(world, router):
    t = Tensor
    with pytest.raises(moe.MoeError) as e:
        moe.decode_layer(t((2, 64), BF), t((4, 64), F32), t((4, 8, 64), BF), t((4, 8, 64), BF), t((4, 64, 8), BF), 2, router=router)
    assert e.value.status == moe.ERR_INVALID_ARG and not calls(world)
