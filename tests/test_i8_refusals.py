"""CPU checks of the entry points of the layer in 8-bit integers: the C ABI refuses
invalid arguments on the host (fake pointers, never dereferenced), empty calls succeed
without a launch, and the binding refuses tensors that it cannot hand on."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_amd import ep

OK, EINVAL, EUNSUP, EWS = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x100000)
OFF2, OFF4, OFF8 = (ctypes.c_void_p(0x100000 + n) for n in (2, 4, 8))


def call(name, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    st = getattr(ep.lib(), name)(*a.values(), None)
    if st:
        assert ep.lib().ep_last_error().startswith(name.encode() + b":")
    return st


DISPATCH = dict(x=FAKE, idx=FAKE, w=None, T=16, H=256, k=2, E=8, R=4, recv=FAKE, scales=FAKE, src=FAKE, rw=None, eoff=FAKE,
                roff=None, row=FAKE, ws=FAKE, wsb=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EUNSUP), (dict(E=9), EINVAL), (dict(E=4096), EUNSUP), (dict(H=0), EINVAL),
    (dict(H=8), EINVAL), (dict(H=24), EINVAL), (dict(x=None), EINVAL), (dict(recv=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(src=None), EINVAL), (dict(eoff=None), EINVAL), (dict(row=None), EINVAL), (dict(x=OFF8), EINVAL), (dict(recv=OFF8), EINVAL),
    (dict(scales=OFF2), EINVAL), (dict(ws=None), EWS), (dict(wsb=16), EWS), (dict(ws=OFF2), EINVAL), (dict(T=2 ** 30), EUNSUP),
])
def test_dispatch(kw, code):
    assert call("ep_dispatch_i8", DISPATCH, kw) == code


CACHED = dict(x=FAKE, row=FAKE, T=16, H=256, k=2, recv=FAKE, scales=FAKE, rows=32)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EUNSUP), (dict(H=8), EINVAL), (dict(H=40), EINVAL),
    (dict(x=None), EINVAL), (dict(row=None), EINVAL), (dict(recv=None), EINVAL), (dict(scales=None), EINVAL), (dict(x=OFF8), EINVAL),
    (dict(recv=OFF4), EINVAL), (dict(scales=OFF2), EINVAL), (dict(T=0), OK), (dict(rows=0, recv=None, scales=None), OK),
])
def test_cached(kw, code):
    assert call("ep_dispatch_i8_cached", CACHED, kw) == code


PADDED = dict(x=FAKE, idx=FAKE, w=None, T=16, H=256, k=2, E=8, cap=4, recv=FAKE, scales=FAKE, count=FAKE, src=FAKE, rw=None,
              slot=FAKE, ws=FAKE, wsb=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(E=0), EINVAL), (dict(cap=0), EINVAL), (dict(E=2048, cap=2 ** 20), EUNSUP),
    (dict(H=24), EINVAL), (dict(x=None), EINVAL), (dict(recv=None), EINVAL), (dict(scales=None), EINVAL), (dict(count=None), EINVAL),
    (dict(src=None), EINVAL), (dict(slot=None), EINVAL), (dict(recv=OFF8), EINVAL), (dict(scales=OFF2), EINVAL), (dict(ws=None), EWS),
    (dict(ws=OFF2), EINVAL),
])
def test_padded(kw, code):
    assert call("ep_dispatch_ll_i8", PADDED, kw) == code


QUANTIZE = dict(x=FAKE, rows=32, H=256, erows=FAKE, E=8, capacity=0, codes=FAKE, scales=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(rows=2 ** 31), EUNSUP), (dict(H=0), EINVAL), (dict(H=24), EINVAL), (dict(E=0), EINVAL),
    (dict(E=2049), EUNSUP), (dict(capacity=-1), EINVAL), (dict(capacity=3), EINVAL), (dict(x=None), EINVAL), (dict(codes=None), EINVAL),
    (dict(scales=None), EINVAL), (dict(x=OFF8), EINVAL), (dict(codes=OFF8), EINVAL), (dict(scales=OFF2), EINVAL), (dict(rows=0), OK),
    (dict(rows=0, erows=None, E=0, capacity=-5, x=None), OK),
])
def test_quantize(kw, code):
    assert call("ep_quantize_i8", QUANTIZE, kw) == code


LINEAR = dict(x=FAKE, xs=FAKE, rows=32, erows=FAKE, capacity=0, w=FAKE, ws=FAKE, E=8, K=256, N=64, epilogue=0, y=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(rows=2 ** 31), EUNSUP), (dict(capacity=-1), EINVAL), (dict(capacity=3), EINVAL), (dict(E=0), EINVAL),
    (dict(E=2049), EUNSUP), (dict(K=64), EINVAL), (dict(K=192), EINVAL), (dict(K=0), EINVAL), (dict(K=(1 << 16) + 128), EUNSUP),
    (dict(N=0), EINVAL), (dict(N=12), EINVAL), (dict(N=2 ** 22 + 8), EUNSUP), (dict(N=2 ** 31 - 8), EUNSUP), (dict(epilogue=2), EINVAL),
    (dict(x=None), EINVAL), (dict(xs=None), EINVAL), (dict(erows=None), EINVAL), (dict(w=None), EINVAL), (dict(ws=None), EINVAL), (dict(y=None), EINVAL),
    (dict(x=OFF8), EINVAL), (dict(xs=OFF2), EINVAL), (dict(w=OFF8), EINVAL), (dict(ws=OFF8), EINVAL), (dict(y=OFF8), EINVAL),
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK),
])
def test_linear(kw, code):
    assert call("ep_expert_linear_i8", LINEAR, kw) == code


MOE = dict(x=FAKE, idx=FAKE, w=FAKE, T=16, H=256, k=2, E=8, F=128, up=FAKE, us=FAKE, down=FAKE, ds=FAKE, out=FAKE, ws=FAKE, wsb=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EUNSUP), (dict(T=257), EUNSUP), (dict(T=2 ** 30, k=1), EUNSUP),
    (dict(T=2 ** 62, k=4), EUNSUP), (dict(E=0), EINVAL), (dict(E=2049), EUNSUP), (dict(H=0), EINVAL), (dict(H=192), EINVAL),
    (dict(F=0), EINVAL), (dict(F=64), EINVAL), (dict(H=65664), EUNSUP), (dict(F=32896), EUNSUP), (dict(idx=None), EINVAL),
    (dict(x=None), EINVAL), (dict(up=None), EINVAL), (dict(us=None), EINVAL), (dict(down=None), EINVAL), (dict(ds=None), EINVAL),
    (dict(out=None), EINVAL), (dict(x=OFF8), EINVAL), (dict(up=OFF8), EINVAL), (dict(us=OFF8), EINVAL), (dict(down=OFF8), EINVAL),
    (dict(ds=OFF8), EINVAL), (dict(out=OFF8), EINVAL), (dict(ws=None), EWS), (dict(wsb=16 * 2 * 132 * 4 - 1), EWS), (dict(ws=OFF8), EINVAL),
    (dict(T=0), OK), (dict(T=0, x=None, idx=None, ws=None, wsb=0), OK),
])
def test_moe(kw, code):
    assert call("ep_moe_i8", MOE, kw) == code


def test_moe_workspace():
    assert ep.ep_moe_i8_workspace_bytes(64, 8, 2048) == 64 * 8 * (2048 + 2048 // 32) * 4
    assert ep.ep_moe_i8_workspace_bytes(65, 8, 2048) == 0 and ep.ep_moe_i8_workspace_bytes(-1, 8, 2048) == 0


def empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


BF, I8, I32, I64 = torch.bfloat16, torch.int8, torch.int32, torch.int64


def test_binding_refuses_what_it_cannot_pass_on():
    x, idx, w = torch.zeros(4, 128).bfloat16(), torch.zeros(4, 2, dtype=I64), torch.zeros(4, 2)
    for fn in (lambda *a: ep.ep_dispatch_i8(*a, 8, 1), lambda *a: ep.ep_dispatch_ll_i8(*a, 8, 3),
               lambda *a: ep.ep_moe_i8(*a, empty(8, 256, 128, dtype=I8), empty(8, 256), empty(8, 128, 128, dtype=I8), empty(8, 128))):
        with pytest.raises(ValueError, match="x must be a device tensor"):
            fn(x, idx, w)
        with pytest.raises(TypeError, match="x must be torch.bfloat16"):
            fn(x.float(), idx, w)
        with pytest.raises(ValueError, match="x must be \\[T, H\\]"):
            fn(x, idx[:3], w)
    with pytest.raises(ValueError, match="token_row"):
        ep.ep_dispatch_i8_cached(x, idx.int()[:3], 8)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        ep.ep_quantize_i8(x.float())
    with pytest.raises(TypeError, match="x_i8 must be torch.int8"):
        ep.ep_expert_linear_i8(x, w, idx, empty(2, 8, 128, dtype=I8), empty(2, 8))
    with pytest.raises(ValueError, match="x_i8 must be \\[rows, K\\]"):
        ep.ep_expert_linear_i8(x[0], w, idx, empty(2, 8, 128, dtype=I8), empty(2, 8))
    with pytest.raises(ValueError, match="x must be \\[T, H\\], up_i8"):
        ep.ep_moe_i8(x, idx, w, empty(256, 128, dtype=I8), empty(8, 256), empty(8, 128, 128, dtype=I8), empty(8, 128))


@pytest.mark.parametrize("v", [2 ** 31, 2 ** 32 + 1, 2 ** 64 + 2, -2 ** 31 - 1])
def test_numbers_past_32_bits(v):
    x, idx = empty(4, 128, dtype=BF), empty(4, 2, dtype=I64)
    for kw in (dict(num_experts=v, num_ranks=1), dict(num_experts=8, num_ranks=v)):
        with pytest.raises(ValueError, match="ep_dispatch_i8.*32-bit"):
            ep.ep_dispatch_i8(x, idx, None, **kw)
    for kw in (dict(num_experts=v, capacity=1), dict(num_experts=8, capacity=v)):
        with pytest.raises(ValueError, match="ep_dispatch_ll_i8.*32-bit"):
            ep.ep_dispatch_ll_i8(x, idx, None, **kw)
    with pytest.raises(ValueError, match="ep_quantize_i8.*32-bit"):
        ep.ep_quantize_i8(x, empty(3, dtype=I32), capacity=v)
    with pytest.raises(ValueError, match="ep_expert_linear_i8.*32-bit"):
        ep.ep_expert_linear_i8(empty(4, 128, dtype=I8), empty(4), empty(3, dtype=I32), empty(2, 8, 128, dtype=I8), empty(2, 8), capacity=v)


@pytest.mark.parametrize("v", [2 ** 31, 2 ** 32 + 16])
def test_sizes_past_32_bits(v):
    with pytest.raises(ValueError, match="ep_dispatch_i8.*32-bit"):
        ep.ep_dispatch_i8(empty(1, v, dtype=BF), empty(1, 2, dtype=I64), None, 8, 1)
    with pytest.raises(ValueError, match="ep_dispatch_i8_cached.*32-bit"):
        ep.ep_dispatch_i8_cached(empty(1, 128, dtype=BF), empty(1, v, dtype=I32), 8)
    with pytest.raises(ValueError, match="ep_quantize_i8.*32-bit"):
        ep.ep_quantize_i8(empty(1, v, dtype=BF))
    for x, w in ((empty(1, v, dtype=I8), empty(2, 8, v, dtype=I8)), (empty(1, 128, dtype=I8), empty(v, 8, 128, dtype=I8)),
                 (empty(1, 128, dtype=I8), empty(2, v, 128, dtype=I8))):
        with pytest.raises(ValueError, match="ep_expert_linear_i8.*32-bit"):
            ep.ep_expert_linear_i8(x, empty(1), empty(3, dtype=I32), w, empty(w.shape[0], w.shape[1]))
    with pytest.raises(ValueError, match="ep_moe_i8.*32-bit"):
        ep.ep_moe_i8(empty(1, 128, dtype=BF), empty(1, 2, dtype=I64), None, empty(v, 256, 128, dtype=I8), empty(v, 256),
                     empty(v, 128, 128, dtype=I8), empty(v, 128))
