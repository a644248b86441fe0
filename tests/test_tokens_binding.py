"""What the token path's binding gives the library, without a GPU: stand-ins for the library, for tensors on several
devices and for the current device note what reaches the entry points."""
import contextlib

import pytest
import torch

import moe_routed_expert_router_gb300 as moe

T, H, K, E, R = 6, 64, 2, 4, 12
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Tensor:
    """A tensor of that shape and type on cuda:<index>, without memory."""

    def __init__(self, shape, dtype, index=0):
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        self.device, self.index, self.streams, self.requires_grad = torch.device("cuda", index), index, [], False

    shape = property(lambda self: self.meta.shape)
    dtype = property(lambda self: self.meta.dtype)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 256 if self.meta.numel() else 0

    def record_stream(self, stream):
        self.streams.append(stream)

    def __getattr__(self, name):          # stride, dim, is_contiguous, element_size
        return getattr(self.meta, name)


class Stream:
    def __init__(self, index):
        self.device, self.device_index, self.cuda_stream = torch.device("cuda", index), index, 7000 + index


class World:
    """The current device, and the calls of the library: (name, arguments, device current at the call)."""

    def __init__(self, monkeypatch):
        self.current, self.calls, self.switches = 0, [], 0
        real = moe.lib()

        class Lib:
            def __getattr__(_, name):
                if name in ("moe_sorted_rows", "moe_rms_norm_backward_workspace", "moe_rms_norm_backward_workspace_for"):
                    return getattr(real, name)

                def call(*args):
                    self.calls.append((name, args, self.current))
                    return moe.OK
                return call

        @contextlib.contextmanager
        def device(index):
            was, self.current = self.current, index
            self.switches += 1
            try:
                yield
            finally:
                self.current = was

        fake = Lib()
        monkeypatch.setattr(moe, "lib", lambda: fake)
        monkeypatch.setattr(moe, "_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(moe, "_devices", 2, raising=False)
        monkeypatch.setattr(moe, "_current_device", lambda: self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, index, stream: 4096)
        monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda p: None)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def every_call(index=0, stream=None, T=T, H=H):
    """Each function of the token path on tensors of cuda:<index>: (name, call, the tensors it is given)."""
    def t(*shape, dtype=BF):
        return Tensor(shape, dtype, index)
    x, r, w, g = t(T, H), t(T, H), t(H), t(T, H)
    rstd, p = t(T, dtype=F32), t(T, K, dtype=F32)
    ids, y, base, scales = t(T, K, dtype=I32), t(R, H), t(T, H), t(T, 4, dtype=F32)
    order = dict(sorted_rows=t(R, dtype=I32), pair_rows=t(T, K, dtype=I32))
    held = list(order.values())
    norm = dict(sum=t(T, H), q=t(T, H, dtype=torch.float8_e4m3fn), scales=t(T, -(-H // 128), dtype=F32), rstd=t(T, dtype=F32))
    back = dict(grad_sum=t(T, H), grad_w=t(H, dtype=F32))
    sort = dict(expert_offsets=t(E + 1, dtype=I32), sorted_rows=t(T * K, dtype=I32), pair_rows=t(T, K, dtype=I32))
    disp = dict(rows=t(R, H), scales=t(R, 4, dtype=F32))
    out, out2 = t(T, H), t(T, H)
    cb = dict(grad_y=t(R, H), grad_w=t(T, K, dtype=F32))
    kw = dict(stream=stream)
    return [
        ("moe_rms_norm", lambda: moe.rms_norm(x, w, residual=r, quant=moe.QUANT_E4M3_128, out=norm, **kw), [x, w, r, *norm.values()]),
        ("moe_rms_norm_backward", lambda: moe.rms_norm_backward(g, x, w, rstd, grad_sum=r, out=back, **kw),
         [g, x, w, rstd, r, *back.values()]),
        ("moe_sort_pairs", lambda: moe.sort_pairs(ids, E, out=sort, **kw), [ids, *sort.values()]),
        ("moe_dispatch", lambda: moe.dispatch(x, order, scales=scales, out=disp, **kw), [x, scales, *held, *disp.values()]),
        ("moe_combine", lambda: moe.combine(y, order, p, base=base, out=out, **kw), [y, p, base, held[1], out]),
        ("moe_combine", lambda: moe.dispatch_backward(y, order, out=out2, **kw), [y, held[1], out2]),
        ("moe_combine_backward", lambda: moe.combine_backward(g, y, order, p, out=cb, **kw), [g, y, p, *held, *cb.values()]),
    ]


@pytest.mark.parametrize("which", range(7))
@pytest.mark.parametrize("given", [False, True])
def test_the_tensors_device_is_current_at_the_call(world, which, given):
    name, call, _ = every_call(1, Stream(1) if given else None)[which]
    call()
    (got, args, current), = world.calls
    assert got == name and current == 1 and args[-1] == (7001 if given else 1001)
    assert world.current == 0
    world.current = 1                                    # no switch where it is current already
    before = world.switches
    call()
    assert world.switches == before and world.calls[-1][2] == 1


@pytest.mark.parametrize("which", range(7))
def test_a_stream_of_another_device_is_refused(world, which):
    _, call, _ = every_call(0, Stream(1))[which]
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.ERR_INVALID_ARG and not world.calls


@pytest.mark.parametrize("which", range(7))
def test_memory_of_the_tensors_is_held_for_a_given_stream(world, which):
    """What a call on another stream reads and writes is recorded there: torch gives freed memory away otherwise."""
    _, call, tensors = every_call(0)[which]
    call()
    assert not any(t.streams for t in tensors)           # the current stream: nothing to record
    stream = Stream(0)
    _, call, tensors = every_call(0, stream)[which]
    call()
    assert all(t.streams == [stream] for t in tensors)


# --------------------------------- sizes that the entry points' 32-bit arguments cannot hold

@pytest.mark.parametrize("size", [dict(T=(1 << 32) + 6), dict(H=(1 << 32) + 64), dict(T=1 << 31)])
@pytest.mark.parametrize("which", range(7))
def test_sizes_past_32_bits_are_refused(world, which, size):
    name, call, _ = every_call(**size)[which]
    if "H" in size and name in ("moe_sort_pairs", "moe_dispatch"):
        pytest.skip("no H, or a row's bytes in 64 bits, of which the library takes 2^31 - 1")
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.ERR_UNSUPPORTED_SHAPE and not world.calls


def test_pairs_a_token_and_scales_past_32_bits_are_refused(world):
    many = (1 << 32) + 2
    order = dict(sorted_rows=Tensor((R,), I32), pair_rows=Tensor((T, many), I32))
    good = dict(sorted_rows=Tensor((R,), I32), pair_rows=Tensor((T, K), I32))
    for call in (lambda: moe.combine(Tensor((R, H), BF), order, out=Tensor((T, H), BF)),
                 lambda: moe.dispatch(Tensor((T, H), BF), order, out=dict(rows=Tensor((R, H), BF))),
                 lambda: moe.dispatch(Tensor((T, H), BF), good, scales=Tensor((T, 1 << 30), F32),
                                      out=dict(rows=Tensor((R, H), BF), scales=Tensor((R, 1 << 30), F32)))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.ERR_UNSUPPORTED_SHAPE and not world.calls


@pytest.mark.parametrize("args", [(10, (1 << 32) + 8), (10, 8 - (1 << 32)), (10, 8, (1 << 32) + 1), (10, 8, 1 - (1 << 32)),
                                  ((1 << 64) + 10, 8)])
def test_sorted_rows_of_sizes_past_32_bits(args):
    with pytest.raises(moe.MoeError) as e:
        moe.sorted_rows(*args)
    assert e.value.status == moe.ERR_UNSUPPORTED_SHAPE


# --------------------------------- tensors that autograd follows

@pytest.mark.parametrize("which,names", [(0, 3), (3, 2), (4, 3), (5, 1)])
def test_tensors_that_require_a_gradient_are_not_taken_in_silence(world, which, names):
    """The results have no history: the forward calls refuse what autograd would follow, unless it is switched off."""
    for i in range(names):
        name, call, tensors = every_call()[which]
        tensors[i].requires_grad = True
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.ERR_INVALID_ARG and "no_grad" in str(e.value) and not world.calls
        with torch.no_grad():
            call()
        (got, _, _), = world.calls
        assert got == name
        world.calls.clear()
