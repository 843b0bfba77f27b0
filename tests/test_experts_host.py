"""Host-side checks of the experts' ops (no GPU needed): every refusal comes
before any HIP call, and the custom ops have fake implementations."""
import ctypes as C

import pytest
import torch

import combine_ep_prepare_amd as ep

# Fake, never dereferenced device addresses (16-byte aligned / misaligned).
P = C.c_void_p(0x10000)
MIS = C.c_void_p(0x10008)
BIG = 1 << 30


def lay(T=16, K=2, E=4, A=8, H=64, cap=96, **kw):
    return ep.Layout(T, K, E, A, H, cap, **kw)


def linear(L, n=64, h=P, nb=BIG, x=P, w=P, o=P):
    return ep.lib.ep_grouped_linear(C.byref(L) if L else None, h, nb, x, w, o, n, None)


def linear_bwd(L, n=64, h=P, nb=BIG, g=P, x=P, w=P, gx=P, gw=P):
    return ep.lib.ep_grouped_linear_bwd(C.byref(L) if L else None, h, nb, g, x, w, gx, gw, n,
                                        None)


def quant(L, n=64, G=32, h=P, nb=BIG, x=P, q=P, s=P, z=P, o=P):
    return ep.lib.ep_grouped_linear_quant(C.byref(L) if L else None, h, nb, x, q, s, z, o, n, G,
                                          None)


def swiglu(L, h=P, nb=BIG, gu=P, o=P):
    return ep.lib.ep_swiglu(C.byref(L) if L else None, h, nb, gu, o, None)


def swiglu_bwd(L, h=P, nb=BIG, g=P, gu=P, o=P):
    return ep.lib.ep_swiglu_bwd(C.byref(L) if L else None, h, nb, g, gu, o, None)


ALL = [linear, linear_bwd, quant, swiglu, swiglu_bwd]


@pytest.mark.parametrize("call", ALL)
def test_layout_and_handle_checks(call):
    L = lay()
    assert call(lay(K=0)) == ep.EP_ERR_SHAPE
    assert call(lay(H=12)) == ep.EP_ERR_SHAPE
    assert call(lay(cap=-1)) == ep.EP_ERR_CAPACITY
    assert call(None) == ep.EP_ERR_NULL
    assert call(L, h=None) == ep.EP_ERR_NULL
    assert call(L, nb=ep.handle_regions(L).maps_bytes - 1) == ep.EP_ERR_HANDLE_SIZE
    assert call(L, h=MIS) == ep.EP_ERR_ALIGN


@pytest.mark.parametrize("call", [linear, linear_bwd, quant])
@pytest.mark.parametrize("n", [-8, 0, 4, 12, (1 << 20) + 8, 1 << 40])
def test_feature_counts(call, n):
    assert call(lay(), n=n) == ep.EP_ERR_SHAPE
    assert call(lay(H=(1 << 20) + 64)) == ep.EP_ERR_SHAPE


@pytest.mark.parametrize("call,names", [
    (linear, ("x", "w", "o")), (linear_bwd, ("g",)), (quant, ("x", "q", "s", "o")),
    (swiglu, ("gu", "o")), (swiglu_bwd, ("g", "gu", "o"))])
def test_required_pointers(call, names):
    for name in names:
        assert call(lay(), **{name: None}) == ep.EP_ERR_NULL, name
        assert call(lay(T=0), **{name: None}) == ep.EP_ERR_NULL, name


@pytest.mark.parametrize("call,names", [
    (linear, ("x", "w", "o")), (linear_bwd, ("g", "x", "w", "gx", "gw")),
    (quant, ("x", "q", "s", "z", "o")), (swiglu, ("gu", "o")), (swiglu_bwd, ("g", "gu", "o"))])
def test_alignment(call, names):
    for name in names:
        assert call(lay(), **{name: MIS}) == ep.EP_ERR_ALIGN, name


def test_weights_are_required_whatever_the_capacity():
    L = lay(cap=0)
    assert linear(L, x=None, w=None, o=None) == ep.EP_ERR_NULL
    assert quant(L, x=None, q=None, o=None) == ep.EP_ERR_NULL
    assert quant(L, x=None, s=None, o=None) == ep.EP_ERR_NULL


def test_backward_outputs_and_their_operands():
    L = lay()
    assert linear_bwd(L, gx=None, gw=None) == ep.EP_ERR_NULL
    assert linear_bwd(L, w=None) == ep.EP_ERR_NULL            # grad_x needs the weight
    assert linear_bwd(L, x=None) == ep.EP_ERR_NULL            # grad_weight needs x
    # a skipped output's operand may be missing: the next check (alignment) is reached
    assert linear_bwd(L, w=None, gx=None, g=MIS) == ep.EP_ERR_ALIGN
    assert linear_bwd(L, x=None, gw=None, g=MIS) == ep.EP_ERR_ALIGN


def test_quant_groups_and_types():
    for G in (0, -32, 16, 48, 96, 256):
        assert quant(lay(H=768), G=G) == ep.EP_ERR_SHAPE
    assert quant(lay(H=96), G=64) == ep.EP_ERR_SHAPE          # the group must divide H
    assert quant(lay(H=64, dtype="fp32"), G=32) == ep.EP_ERR_SHAPE
    assert quant(lay(H=64), G=64, x=MIS) == ep.EP_ERR_ALIGN
    assert quant(lay(H=64), G=64, z=None, x=MIS) == ep.EP_ERR_ALIGN


def test_binding_refuses_wrong_tensors():
    L = lay()
    h = torch.empty(ep.handle_mem_size(L), dtype=torch.uint8)
    x = torch.zeros(96, 64, dtype=torch.bfloat16)
    w = torch.zeros(4, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                           # weight not [E,N,H]
        ep.grouped_linear(L, h, x, w[0], x)
    with pytest.raises(ValueError):                           # not GPU tensors
        ep.grouped_linear(L, h, x, w, x)
    with pytest.raises(ValueError):
        ep.grouped_linear_bwd(L, h, x[0], x, w, x, w)
    with pytest.raises(ValueError):                           # 5 groups do not divide H = 64
        ep.grouped_linear_quant(L, h, x, w, torch.zeros(4, 64, 5), None, x)
    with pytest.raises(ValueError):
        ep.swiglu(L, h, x, x)


def test_autograd_refusals_on_cpu():
    from combine_ep_prepare_amd import autograd as epa

    class Routing:                                            # never reached past the checks
        pass

    x = torch.zeros(96, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError):
        epa.grouped_linear(x[0], x, Routing())
    with pytest.raises(ValueError):
        epa.swiglu(x[0], Routing())
    with pytest.raises(RuntimeError, match="no backward"):
        epa.grouped_linear_quant(x, x, x, Routing())


def test_custom_ops_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode

    import combine_ep_prepare_amd.custom_ops as co
    L = lay()
    ll = co.layout_list(L)
    with FakeTensorMode():
        h = torch.empty(ep.handle_mem_size(L), dtype=torch.uint8)
        x = torch.empty(96, 64, dtype=torch.float16)
        w = torch.empty(4, 48, 64, dtype=torch.float16)
        out = co.grouped_linear(x, w, h, ll)
        assert out.shape == (96, 48) and out.dtype == torch.float16
        gx, gw = co.grouped_linear_bwd(out, x, w, h, ll)
        assert gx.shape == x.shape and gw.shape == w.shape
        act = co.swiglu(out, h, ll)
        assert act.shape == (96, 24)
        assert co.swiglu_bwd(act, out, h, ll).shape == out.shape
        q = torch.empty(4, 48, 32, dtype=torch.uint8)
        s = torch.empty(4, 48, 2, dtype=torch.float16)
        assert co.grouped_linear_quant(x, q, s, None, h, ll).shape == (96, 48)
