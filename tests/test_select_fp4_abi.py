"""CPU-side checks of routing from logits and of the 4-bit expert calls: every
bad argument is refused on the host, by the C ABI with its status and by the
binding with an exception, before anything reaches the GPU."""
import ctypes
import inspect

import pytest
import torch

import grouped_top_routing_amd as gtr
from grouped_top_routing_amd import _lib as L

# fake, never-dereferenced device addresses, far apart
A, B, C, D, P = (ctypes.c_void_p(i << 40) for i in range(1, 6))
MIS, ODD = ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10001)
INVALID, UNSUPPORTED, WORKSPACE = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE
BIG = 1 << 39


def _sel(T=64, E=256, groups=8, kept=4, best=2, k=8, score=1, renorm=1, dt=1):
    return L.MoeSelectConfig(T, E, groups, kept, best, k, score, renorm, dt)


def _select(c, z=A, bias=None, ids=B, w=C):
    return gtr.lib().moe_select(ctypes.byref(c) if c else None, z, bias, ids, w, None)


def _backward(c, z=A, ids=B, g=C, load=None, gl=None, out=D):
    return gtr.lib().moe_select_backward(ctypes.byref(c) if c else None, z, ids, g, load, gl, out,
                                         None)


def _balance(c, z=A, ids=B, coef=0.1, loss=C, load=D, ws=P, nb=BIG):
    return gtr.lib().moe_balance_loss(ctypes.byref(c) if c else None, z, ids, coef, loss, load, ws,
                                      nb, None)


def _route_select(c, s, x=A, wr=B, bias=None, ids=C, w=D, z=None, ws=P, nb=BIG):
    return gtr.lib().moe_route_select(ctypes.byref(c) if c else None,
                                      ctypes.byref(s) if s else None, x, wr, bias, ids, w, z, ws,
                                      nb, None)


@pytest.mark.parametrize("call", [_select, _backward, _balance])
def test_selection_checks_its_configuration(call):
    assert call(None) == INVALID
    assert call(_sel(T=0)) == L.MOE_OK
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(score=2), dict(score=-1), dict(dt=2),
               dict(dt=-1), dict(renorm=2)):
        assert call(_sel(**{"T": 0, **kw})) == INVALID, kw
    for kw in (dict(E=1025, groups=1, kept=1), dict(k=33, groups=1, kept=1),
               dict(T=1 << 26)):
        assert call(_sel(**{"T": 0, **kw})) == UNSUPPORTED, kw


def test_selection_checks_its_groups():
    for kw in (dict(groups=0), dict(kept=0), dict(kept=9), dict(groups=7), dict(best=0),
               dict(best=3), dict(groups=64, kept=1, k=5)):
        assert _select(_sel(T=0, **kw)) == INVALID, kw
        assert _backward(_sel(T=0, **kw)) == L.MOE_OK  # reads no groups
    assert _select(_sel(T=0, groups=128, kept=8)) == UNSUPPORTED
    assert _select(_sel(T=0, E=1024, groups=64, kept=64, k=32)) == L.MOE_OK
    assert _select(_sel(T=0, E=1, groups=1, kept=1, k=1)) == L.MOE_OK


def test_selection_checks_its_pointers():
    c = _sel(T=0)
    for kw in (dict(z=None), dict(ids=None), dict(w=None), dict(z=ODD), dict(bias=ODD),
               dict(ids=ODD), dict(w=ODD)):
        assert _select(c, **kw) == INVALID, kw
    assert _select(_sel(T=0, dt=0), z=ctypes.c_void_p(0x10002)) == L.MOE_OK  # bf16 elements
    for kw in (dict(z=None), dict(ids=None), dict(out=None), dict(g=None), dict(gl=P),
               dict(z=ODD), dict(out=ODD), dict(g=ODD), dict(load=ODD), dict(load=P, gl=ODD)):
        assert _backward(c, **kw) == INVALID, kw
    assert _backward(c, g=None, load=P) == L.MOE_OK
    for kw in (dict(z=None), dict(ids=None), dict(loss=None), dict(load=None), dict(z=ODD),
               dict(loss=ODD), dict(load=ODD), dict(coef=float("inf")), dict(coef=float("nan"))):
        assert _balance(c, **kw) == INVALID, kw
    c = _sel(T=64)
    n = ctypes.c_size_t(0)
    assert gtr.lib().moe_balance_workspace_bytes(ctypes.byref(c), ctypes.byref(n)) == 0 and n.value
    assert gtr.lib().moe_balance_workspace_bytes(ctypes.byref(c), None) == INVALID
    assert gtr.lib().moe_balance_workspace_bytes(None, ctypes.byref(n)) == INVALID
    assert _balance(c, ws=None) == WORKSPACE and _balance(c, nb=n.value - 1) == WORKSPACE
    assert _balance(c, ws=MIS) == INVALID


def test_selection_refuses_overlapping_memory():
    at = lambda p, n: ctypes.c_void_p(p.value + n)
    c = _sel(T=64)
    size, slots = 64 * 256 * 4, 64 * 8 * 4
    assert _select(c, ids=at(A, size - 4)) == INVALID
    assert _select(c, ids=B, w=at(B, slots - 4)) == INVALID
    assert _select(c, bias=at(C, 8)) == INVALID
    assert _backward(c, out=A) == INVALID and _backward(c, out=at(A, 4 - size)) == INVALID
    assert _backward(c, g=at(D, size - 4)) == INVALID
    assert _backward(c, load=P, gl=at(D, 16)) == INVALID
    assert _balance(c, loss=at(D, 12)) == INVALID
    assert _balance(c, load=at(A, 0)) == INVALID
    assert _balance(c, ws=at(A, 16)) == INVALID


def test_route_select_checks_its_arguments():
    c, s = gtr.make_config(0, 512, 128), _sel(T=0)
    assert _route_select(c, s) == L.MOE_OK
    assert _route_select(None, s) == INVALID and _route_select(c, None) == INVALID
    for kw in (dict(T=1), dict(E=128), dict(dt=0), dict(score=3), dict(kept=0)):
        assert _route_select(c, _sel(**{"T": 0, **kw})) == INVALID, kw
    assert _route_select(gtr.make_config(0, 500, 128), s) == UNSUPPORTED
    assert _route_select(gtr.make_config(0, 512, 128, num_experts=128), _sel(T=0, E=128)) == UNSUPPORTED
    for kw in (dict(x=None), dict(wr=None), dict(ids=None), dict(w=None), dict(x=MIS),
               dict(wr=MIS), dict(z=ODD), dict(bias=ODD)):
        assert _route_select(c, s, **kw) == INVALID, kw
    c, s = gtr.make_config(64, 512, 128, weight_layout=gtr.LAYOUT_FP4_PACKED), _sel()
    assert _route_select(c, s, ws=None) == WORKSPACE
    assert _route_select(c, s, z=A) == INVALID and _route_select(c, s, z=P) == INVALID


# ---------------------------------------------------------------------------
def _cfg(T=64, H=512, I=256, layout=None, **kw):
    return gtr.make_config(T, H, I, weight_layout=gtr.LAYOUT_FP4_PACKED if layout is None else layout,
                           **kw)


def _ffn(c, x=A, src=A, off=A, qg=A, sg=A, qd=A, sd=A, y=A, ws=A, nb=BIG):
    return gtr.lib().moe_expert_ffn_fp4(ctypes.byref(c), x, src, off, qg, sg, qd, sd, y, ws, nb, None)


def _gate_up(c, x=A, src=A, off=A, q=A, s=A, h=A, ws=A, nb=BIG):
    return gtr.lib().moe_expert_gate_up_fp4(ctypes.byref(c), x, src, off, q, s, h, ws, nb, None)


def _down(c, h=A, off=A, q=A, s=A, y=A, ws=A, nb=BIG):
    return gtr.lib().moe_expert_down_fp4(ctypes.byref(c), h, off, q, s, y, ws, nb, None)


def _layer(c, x=A, wr=A, bias=None, qg=A, sg=A, qd=A, sd=A, out=A, ids=None, w=None, ws=A, nb=BIG):
    return gtr.lib().moe_layer_forward_fp4(ctypes.byref(c), x, wr, bias, qg, sg, qd, sd, out, ids,
                                           w, ws, nb, None)


@pytest.mark.parametrize("call", [_ffn, _gate_up, _down, _layer])
def test_fp4_calls_check_layout_configuration_and_pointers(call):
    assert call(_cfg(T=0)) == L.MOE_OK
    for layout in (0, 1, 2, 3, 5, -1):
        assert call(_cfg(T=0, layout=layout)) == INVALID, layout
    assert call(_cfg(T=-1)) == INVALID
    assert call(_cfg(T=0, H=500)) == UNSUPPORTED and call(_cfg(T=0, I=100)) == UNSUPPORTED
    assert call(_cfg(T=1 << 28)) == UNSUPPORTED
    assert call(_cfg(T=0, H=1 << 16, I=1 << 15)) == L.MOE_OK
    assert call(_cfg(T=0, H=1 << 16, I=1 << 16)) == UNSUPPORTED  # an expert past 32 bits
    assert call(_cfg(T=0, H=1 << 23)) == UNSUPPORTED and call(_cfg(T=0, I=1 << 23)) == UNSUPPORTED
    assert call(_cfg(), nb=16) == WORKSPACE and call(_cfg(), ws=None) == WORKSPACE
    names = [n for n in inspect.signature(call).parameters if n not in ("c", "nb", "ws")]
    for n in names:
        if n not in ("bias", "ids", "w"):
            assert call(_cfg(T=0), **{n: None}) == INVALID, n
        assert call(_cfg(T=0), **{n: ODD}) == INVALID, n
        if n not in ("src", "off", "bias", "ids", "w"):
            assert call(_cfg(T=0), **{n: MIS}) == INVALID, n


@pytest.mark.parametrize("call,written", [(_ffn, "y"), (_gate_up, "h"), (_down, "y")])
def test_fp4_calls_refuse_overlapping_memory(call, written):
    at = lambda n: ctypes.c_void_p(n << 44)
    names = [n for n in inspect.signature(call).parameters if n not in ("c", "nb")]
    apart = {n: at(i + 1) for i, n in enumerate(names)}
    for n in names:
        for out in {written, "ws"} - {n}:
            assert call(_cfg(), **{**apart, n: apart[out]}) == INVALID, (n, out)
            assert call(_cfg(T=0), **{**apart, n: apart[out]}) == L.MOE_OK
    inside = ctypes.c_void_p(apart[written].value + 64 * 8 * 256 * 2 - 16)
    assert call(_cfg(), **{**apart, "off": inside}) == INVALID


def test_bf16_and_fp8_calls_refuse_the_fp4_layout():
    c = ctypes.byref(_cfg(T=0))
    assert gtr.lib().moe_expert_down(c, A, A, A, A, A, BIG, None) == INVALID
    assert gtr.lib().moe_expert_down_fp8(c, A, A, A, A, A, A, BIG, None) == INVALID
    for entry in (gtr.ENTRY_EXPERT_FFN, gtr.ENTRY_EXPERT_STAGE, gtr.ENTRY_LAYER):
        assert gtr.workspace_bytes(_cfg(), entry) > 0


@pytest.mark.parametrize("T", [0, 1, 17, 128, 4096, 100000, 1 << 27])
def test_fp4_workspaces_hold_every_tile(T):
    """The plan has room for the rows of T * k pairs cut at any m-tile height the
    calls use (at least 16 rows) over 256 experts, as far as pairs go round."""
    n = gtr.workspace_bytes(_cfg(T=T, H=5120, I=2560), gtr.ENTRY_EXPERT_STAGE)
    assert n >= 5 * 4 * min(256, T * 8)
    assert n <= 4 * 70 * (T * 8 // 16 + 260) + 4096


def test_fp4_weights_check_their_arrays():
    lib, c = gtr.lib(), ctypes.byref(gtr.make_config(0, 512, 256))
    q = lambda *a: lib.moe_quantize_fp4(c, *a, None)
    assert q(None, None, None, None, None, None) == L.MOE_OK
    for i in range(3):
        gu = [A, B, C]
        for bad in (None, MIS):
            gu[i] = bad
            assert q(gu[0], None, gu[1], gu[2], None, None) == INVALID
            assert q(None, gu[0], None, None, gu[1], gu[2]) == INVALID
    assert q(A, None, ctypes.c_void_p(A.value + 64), C, None, None) == INVALID
    assert q(A, None, B, ctypes.c_void_p(B.value + 64), None, None) == INVALID
    assert q(A, B, C, D, C, P) == INVALID  # one output twice
    assert lib.moe_quantize_fp4(ctypes.byref(gtr.make_config(0, 512, 100)), A, None, B, C, None,
                                None, None) == UNSUPPORTED
    big = ctypes.byref(gtr.make_config(0, 1 << 16, 1 << 16))
    assert lib.moe_quantize_fp4(big, None, None, None, None, None, None, None) == UNSUPPORTED
    assert lib.moe_pack_fp4(big, *[None] * 8, None) == UNSUPPORTED
    p = lambda *a: lib.moe_pack_fp4(c, *a, None)
    assert p(*[None] * 8) == L.MOE_OK
    assert p(A, B, None, None, C, None, None, None) == INVALID
    assert p(A, None, None, None, C, D, None, None) == INVALID
    assert p(A, B, None, None, A, D, None, None) == INVALID
    assert p(None, None, A, B, None, None, C, MIS) == INVALID


# ---------------------------------------------------------------------------
def test_binding_refuses_what_the_calls_cannot_take():
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    i = torch.int32
    for call in (lambda: gtr.select(z(2, 8)),
                 lambda: gtr.balance_loss(z(2, 8), z(2, 1, dtype=i)),
                 lambda: gtr.select_backward(z(2, 8), z(2, 1, dtype=i), z(2, 1)),
                 lambda: gtr.route_select(z(2, 256, dtype=torch.bfloat16), z(256, 256)),
                 lambda: gtr.quantize_fp4(z(256, 256, 256, dtype=torch.bfloat16),
                                          z(256, 256, 128, dtype=torch.bfloat16)),
                 lambda: gtr.pack_fp4(*(z(256, 256, n, dtype=torch.uint8) for n in (128, 8, 64, 4)))):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        gtr.select(z(2, 8, dtype=torch.float16))
    with pytest.raises(TypeError, match="torch.Tensor"):
        gtr.select([1.0])
    with pytest.raises(ValueError, match=r"\(T, E\)"):
        gtr.balance_loss(z(8), z(2, 1, dtype=i))
    with pytest.raises(TypeError, match="topk_ids"):
        gtr._select._need_ids(z(8, dtype=i), 8, None)
    with pytest.raises(ValueError, match="score must be one of"):
        gtr._select._config(1, 8, 2, "tanh", True, torch.float32)


@pytest.mark.parametrize("name", ["quantize_fp4", "pack_fp4", "expert_ffn_fp4", "expert_gate_up_fp4",
                                  "expert_down_fp4", "layer_forward_fp4"])
def test_fp4_calls_run_on_their_tensors_device(name):
    fn = getattr(gtr, name)
    assert inspect.unwrap(fn) is not fn and inspect.unwrap(fn).__name__ == name


def test_entry_points_are_declared_and_exported():
    import os
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                               "include", "beam_moe.h")).read()
    for name in ("moe_select", "moe_route_select", "moe_balance_workspace_bytes",
                 "moe_balance_loss", "moe_select_backward", "moe_quantize_fp4", "moe_pack_fp4",
                 "moe_expert_ffn_fp4", "moe_expert_gate_up_fp4", "moe_expert_down_fp4",
                 "moe_layer_forward_fp4"):
        assert name + "(" in header and name in L.EXPORTS and getattr(gtr.lib(), name)
