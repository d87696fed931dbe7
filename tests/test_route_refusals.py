"""CPU checks of the routing, combine-gradient and 4-bit product entry points:
the C ABI refuses invalid arguments on the host (fake pointers, never
dereferenced), empty calls succeed without a launch, and the Python binding
refuses tensors that it cannot hand on."""
import ctypes

import pytest
import torch

from combine_get_dispatch_02_amd import ep

OK, EINVAL, EUNSUP = 0, 1, 2
FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100001)


def call(name, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    st = getattr(ep.lib(), name)(*a.values(), None)
    if st:
        assert ep.lib().ep_last_error().startswith(name.encode() + b":")
    return st


ROUTE = dict(logits=FAKE, type=0, bias=None, T=16, E=64, k=4, score=0, groups=4, topk_groups=2, group_top=2, renorm=1,
             scale=1.0, idx=FAKE, w=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=4096), EUNSUP), (dict(k=0), EINVAL), (dict(k=65), EUNSUP),
    (dict(type=3), EINVAL), (dict(type=-1), EINVAL), (dict(score=2), EINVAL), (dict(groups=0), EINVAL),
    (dict(groups=3), EINVAL), (dict(groups=128, E=256), EUNSUP), (dict(topk_groups=0), EINVAL),
    (dict(topk_groups=5), EINVAL), (dict(group_top=0), EINVAL), (dict(group_top=3), EINVAL), (dict(k=33), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(logits=None), EINVAL),
    (dict(idx=None), EINVAL), (dict(w=None), EINVAL), (dict(logits=ODD), EINVAL),
    (dict(logits=ctypes.c_void_p(0x100002)), EINVAL), (dict(logits=ODD, type=1), EINVAL), (dict(T=2 ** 29), EUNSUP),
    (dict(T=2 ** 62), EUNSUP), (dict(T=0), OK), (dict(T=0, logits=None, idx=None, w=None), OK),
])
def test_route(kw, code):
    assert call("ep_route", ROUTE, kw) == code


BACK = dict(logits=FAKE, type=0, idx=FAKE, g=FAKE, T=16, E=64, k=4, score=0, renorm=1, scale=1.0, out=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=2049), EUNSUP), (dict(k=0), EINVAL), (dict(k=65), EUNSUP),
    (dict(type=7), EINVAL), (dict(score=-1), EINVAL), (dict(scale=float("-inf")), EINVAL), (dict(logits=None), EINVAL),
    (dict(idx=None), EINVAL), (dict(g=None), EINVAL), (dict(out=None), EINVAL),
    (dict(out=ctypes.c_void_p(0x100002)), EINVAL), (dict(out=ODD, type=2), EINVAL), (dict(T=2 ** 30), EUNSUP),
    (dict(T=0), OK),
])
def test_route_backward(kw, code):
    assert call("ep_route_backward", BACK, kw) == code


COMBINE = dict(g=FAKE, y=FAKE, rows=32, row=FAKE, w=FAKE, T=16, H=256, k=2, dy=FAKE, dw=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=65), EUNSUP), (dict(H=4), EINVAL),
    (dict(H=20), EINVAL), (dict(H=0), EINVAL), (dict(g=None), EINVAL), (dict(y=None), EINVAL), (dict(row=None), EINVAL),
    (dict(dy=None, dw=None), EINVAL), (dict(g=ctypes.c_void_p(0x100008)), EINVAL),
    (dict(y=ctypes.c_void_p(0x100008)), EINVAL), (dict(dy=ctypes.c_void_p(0x100004)), EINVAL),
    (dict(T=2 ** 30), EUNSUP), (dict(T=0), OK), (dict(T=0, dy=None, dw=None), OK),
    (dict(rows=0, y=None, dy=None, dw=None), OK), (dict(rows=0, dw=None), OK),
])
def test_combine_backward(kw, code):
    assert call("ep_combine_backward", COMBINE, kw) == code


W4 = dict(x=FAKE, rows=32, erows=FAKE, capacity=0, codes=FAKE, scales=FAKE, E=8, K=256, N=64, epilogue=0, y=FAKE)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(rows=2 ** 31), EUNSUP), (dict(capacity=-1), EINVAL), (dict(capacity=3), EINVAL),
    (dict(E=0), EINVAL), (dict(E=2049), EUNSUP), (dict(K=64), EINVAL), (dict(K=192), EINVAL), (dict(K=0), EINVAL), (dict(K=2 ** 23), EUNSUP),
    (dict(N=0), EINVAL), (dict(N=12), EINVAL), (dict(N=2 ** 31 - 8), EUNSUP), (dict(epilogue=2), EINVAL),
    (dict(x=None), EINVAL), (dict(erows=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(y=None), EINVAL), (dict(x=ctypes.c_void_p(0x100008)), EINVAL), (dict(codes=ctypes.c_void_p(0x100008)), EINVAL),
    (dict(scales=ctypes.c_void_p(0x100002)), EINVAL), (dict(y=ctypes.c_void_p(0x100008)), EINVAL),
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK),
])
def test_expert_linear_w4(kw, code):
    assert call("ep_expert_linear_w4", W4, kw) == code


def test_binding_refuses_what_it_cannot_pass_on():
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route(l, 2)
    with pytest.raises(TypeError, match="logits must be one of"):
        ep.ep_route(l.double(), 2)
    with pytest.raises(TypeError, match="logits must be one of"):
        ep.ep_route_backward(l.int(), l.long(), l)
    with pytest.raises(TypeError, match="grad_out must be torch.bfloat16"):
        ep.ep_combine_backward(l, None, l.int(), None)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        ep.ep_expert_linear_w4(l, l.int(), l, l)
