"""CPU-side checks of the training calls: every bad argument is refused on the
host, by the C ABI with its status and by the binding with an exception, before
anything reaches the GPU."""
import ctypes

import pytest
import torch

import grouped_top_routing_amd as gtr
from grouped_top_routing_amd import _lib as L

# fake, never-dereferenced device addresses
A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10004)
ODD = ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED


def _cfg(T=64, H=256, topk=8, **kw):
    return gtr.make_config(T, H, 128, num_groups=1, topk_groups=1, topk=topk, **kw)


def _dispatch(c, dt=0, x=A, dst=A, w=None, out=A):
    return gtr.lib().moe_dispatch(ctypes.byref(c) if c else None, dt, x, dst, w, out, None)


def _dispatch_backward(c, dt=0, g=A, dst=A, w=None, x=None, gx=A, gw=None):
    return gtr.lib().moe_dispatch_backward(ctypes.byref(c), dt, g, dst, w, x, gx, gw, None)


def _combine_rows(c, dt=0, y=A, dst=A, w=A, out=A):
    return gtr.lib().moe_combine_rows(ctypes.byref(c), dt, y, dst, w, out, None)


def _combine_backward(c, dt=0, g=A, y=A, dst=A, w=A, gy=A, gw=A):
    return gtr.lib().moe_combine_backward(ctypes.byref(c), dt, g, y, dst, w, gy, gw, None)


@pytest.mark.parametrize("call", [_dispatch, _dispatch_backward, _combine_rows, _combine_backward])
def test_row_calls_check_the_configuration(call):
    zero = _cfg(T=0, H=7, topk=3)
    assert call(zero) == L.MOE_OK  # any width; nothing to do
    assert call(zero, dt=2) == INVALID and call(zero, dt=-1) == INVALID
    assert call(_cfg(T=-1)) == INVALID
    assert call(_cfg(H=0)) == INVALID
    assert call(_cfg(topk=0)) == INVALID
    assert call(_cfg(topk=9)) == UNSUPPORTED
    assert call(_cfg(H=(1 << 28) + 1)) == UNSUPPORTED
    assert call(_cfg(T=1 << 28)) == UNSUPPORTED
    assert call(_cfg(T=1 << 62)) == UNSUPPORTED
    assert call(_cfg(routed_scaling=float("inf"))) == INVALID


def test_row_calls_check_their_pointers():
    c = _cfg(T=0)
    assert _dispatch(None) == INVALID
    for kw in (dict(x=None), dict(dst=None), dict(out=None), dict(x=MIS), dict(out=MIS),
               dict(dst=ODD), dict(w=ODD)):
        assert _dispatch(c, **kw) == INVALID, kw
    for kw in (dict(g=None), dict(dst=None), dict(gx=None), dict(g=MIS), dict(gx=MIS),
               dict(w=A, x=MIS, gw=A), dict(w=ODD), dict(x=A), dict(gw=A), dict(w=A, x=A),
               dict(w=A, gw=A), dict(x=A, gw=A), dict(w=A, x=A, gw=ODD)):
        assert _dispatch_backward(c, **kw) == INVALID, kw
    assert _dispatch_backward(c, w=A, x=A, gw=A) == L.MOE_OK
    for kw in (dict(y=None), dict(dst=None), dict(w=None), dict(out=None), dict(y=MIS),
               dict(out=MIS), dict(w=ODD), dict(dst=ODD)):
        assert _combine_rows(c, **kw) == INVALID, kw
    for kw in (dict(g=None), dict(dst=None), dict(gy=None, gw=None), dict(y=None),
               dict(w=None), dict(g=MIS), dict(y=MIS), dict(gy=MIS), dict(gw=ODD), dict(w=ODD)):
        assert _combine_backward(c, **kw) == INVALID, kw
    assert _combine_backward(c, y=None, gw=None) == L.MOE_OK
    assert _combine_backward(c, w=None, gy=None) == L.MOE_OK


def _route_logits(c, x=A, wr=A, bias=None, replay=0, ids=A, w=A, z=A, ws=A, nb=1 << 40):
    return gtr.lib().moe_route_logits(ctypes.byref(c), x, wr, bias, replay, ids, w, z, ws, nb, None)


def _route_backward(c, x=A, wr=A, ids=A, z=A, g=A, src=A, off=A, add=None, acc=0, gw=A, gx=A,
                    ws=A, nb=1 << 40):
    return gtr.lib().moe_route_backward(ctypes.byref(c), x, wr, ids, z, g, src, off, add, acc, gw,
                                        gx, ws, nb, None)


def test_route_calls_check_their_arguments():
    c = _cfg(T=0)
    assert _route_logits(c) == L.MOE_OK and _route_logits(c, replay=1) == L.MOE_OK
    for kw in (dict(x=None), dict(wr=None), dict(ids=None), dict(w=None), dict(z=None),
               dict(replay=2), dict(x=MIS), dict(wr=MIS), dict(z=ODD), dict(bias=ODD)):
        assert _route_logits(c, **kw) == INVALID, kw
    assert _route_backward(c) == L.MOE_OK
    assert _route_backward(c, gx=None) == L.MOE_OK
    assert _route_backward(c, add=A, acc=1) == L.MOE_OK
    for kw in (dict(x=None), dict(wr=None), dict(ids=None), dict(z=None), dict(g=None),
               dict(src=None), dict(off=None), dict(gw=None), dict(add=A, gx=None), dict(acc=2),
               dict(acc=-1), dict(x=MIS), dict(wr=MIS), dict(gw=MIS), dict(gx=MIS), dict(add=MIS),
               dict(ids=ODD), dict(z=ODD), dict(g=ODD), dict(src=ODD), dict(off=ODD)):
        assert _route_backward(c, **kw) == INVALID, kw
    for call in (_route_logits, _route_backward):
        assert call(_cfg(H=320)) == UNSUPPORTED
        assert call(_cfg(num_experts=128)) == UNSUPPORTED
        assert call(_cfg(T=-1)) == INVALID


def test_route_backward_checks_its_workspace():
    c = _cfg(T=4096, H=512)
    need = gtr.workspace_bytes(c, gtr.ENTRY_ROUTE_BACKWARD)
    assert need > 4096 * 8 * 4
    assert _route_backward(c, nb=need - 1) == L.MOE_ERR_WORKSPACE
    assert _route_backward(c, ws=None, nb=need) == L.MOE_ERR_WORKSPACE
    assert _route_backward(c, ws=MIS, nb=need) == INVALID
    # a grid of 2^32 threads or more
    assert _route_backward(_cfg(T=(1 << 31) // 8 - 1, H=256 * 64)) == UNSUPPORTED
    # small batches need none
    assert gtr.workspace_bytes(_cfg(T=128, H=5120), gtr.ENTRY_ROUTE_BACKWARD) == 0
    assert gtr.workspace_bytes(_cfg(T=129, H=5120), gtr.ENTRY_ROUTE_BACKWARD) > 129 * 64


# ---------------------------------------------------------------------------
def _opt(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0,
                step=1)
    base.update(kw)
    return L.MoeAdamw(**base)


def _tensor(**kw):
    base = dict(param=0x10000, grad=0x20000, m=0x30000, v=0x40000, n=100,
                param_dtype=gtr.DTYPE_FP32, grad_dtype=gtr.DTYPE_FP32, state_bits=32)
    base.update(kw)
    return L.MoeAdamwTensor(**base)


def _step(opt, *tensors):
    arr = (L.MoeAdamwTensor * max(1, len(tensors)))(*tensors)
    return gtr.lib().moe_adamw_step(ctypes.byref(opt) if opt else None, arr, len(tensors), None)


def test_adamw_checks_its_hyperparameters():
    empty = _tensor(n=0)
    nan, inf = float("nan"), float("inf")
    assert _step(_opt()) == L.MOE_OK and _step(_opt(), empty) == L.MOE_OK
    for kw in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1),
               dict(beta2=1.0), dict(beta2=nan), dict(eps=-1e-8), dict(eps=nan),
               dict(weight_decay=-1.0), dict(grad_scale=nan), dict(grad_scale=inf), dict(step=0),
               dict(step=-3), dict(step_dev=0x10004), dict(lr_dev=0x10002),
               dict(grad_scale_dev=0x10001)):
        assert _step(_opt(**kw), empty) == INVALID, kw
    assert _step(_opt(step=0, step_dev=0x10008), empty) == L.MOE_OK
    assert _step(None) == INVALID
    assert gtr.lib().moe_adamw_step(ctypes.byref(_opt()), None, 1, None) == INVALID
    assert gtr.lib().moe_adamw_step(ctypes.byref(_opt()), None, -1, None) == INVALID
    assert gtr.lib().moe_adamw_step(ctypes.byref(_opt()), None, 0, None) == L.MOE_OK


def test_adamw_checks_its_tensors():
    scales = dict(m_scale=0x50001, v_scale=0x60003)  # of any alignment
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1),
               dict(param=0x10004), dict(grad=0x20008), dict(m=0x30002), dict(v=0x40001),
               dict(param_dtype=2), dict(grad_dtype=-1), dict(state_bits=16),
               dict(master=0x70000), dict(param_dtype=gtr.DTYPE_BF16),
               dict(param_dtype=gtr.DTYPE_BF16, master=0x70004), dict(state_bits=8),
               dict(state_bits=8, m_scale=0x50000), dict(**scales)):
        assert _step(_opt(), _tensor(**kw)) == INVALID, kw
        assert _step(_opt(), _tensor(n=0), _tensor(**kw)) == INVALID, kw
    assert _step(_opt(), _tensor(n=1 << 34)) == UNSUPPORTED


def test_binding_refuses_tensors_that_are_not_on_a_device():
    f, b, i = torch.float32, torch.bfloat16, torch.int32
    z = lambda *s, dtype=f: torch.zeros(*s, dtype=dtype)
    dst, w = z(16, dtype=i), z(2, 8)
    for call in (lambda: gtr.dispatch(z(2, 4), dst),
                 lambda: gtr.dispatch_backward(z(16, 4), dst),
                 lambda: gtr.combine(z(16, 4), dst, w),
                 lambda: gtr.combine_backward(z(2, 4), z(16, 4), dst, w),
                 lambda: gtr.route_backward(z(2, 256, dtype=b), z(256, 256), z(2, 8, dtype=i), w,
                                            w, dst, z(257, dtype=i)),
                 lambda: gtr.AdamW([z(4)])):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_binding_refuses_wrong_types_and_shapes():
    f, i = torch.float32, torch.int32
    dst = torch.zeros(16, dtype=i)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        gtr.dispatch(torch.zeros(2, 4, dtype=torch.float16), dst)
    with pytest.raises(TypeError, match="torch.Tensor"):
        gtr.dispatch([1.0], dst)
    with pytest.raises(ValueError, match=r"\(T \* 3,\)"):
        gtr.dispatch(torch.zeros(2, 4), dst, topk=3)
    with pytest.raises(ValueError, match=r"\(T \* 8,\)"):
        gtr.dispatch_backward(torch.zeros(16, 4), dst.view(2, 8))
    with pytest.raises(ValueError, match="no gradient"):
        gtr.combine_backward(torch.zeros(2, 4), None, dst, torch.zeros(2, 8), need_grad_y=False,
                             need_grad_w=False)
    with pytest.raises(TypeError, match="topk_w"):
        gtr.combine_backward(torch.zeros(2, 4), None, dst, torch.zeros(16))
    with pytest.raises(ValueError, match="no parameters"):
        gtr.AdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        gtr.AdamW([torch.zeros(4)], state_bits=4)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        gtr.AdamW([torch.zeros(4, dtype=torch.float16)])
