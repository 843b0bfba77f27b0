"""Host-side checks of the norm, the 8-bit ops and the layer for a few tokens (no
GPU needed): every refusal comes before any HIP call."""
import ctypes as C

import pytest
import torch

import combine_ep_prepare_amd as ep

# Fake, never dereferenced device addresses (16-byte aligned / misaligned).
P = C.c_void_p(0x10000)
MIS = C.c_void_p(0x10008)
BIG = 1 << 40


def lay(T=16, K=2, E=4, A=8, H=64, cap=96, **kw):
    return ep.Layout(T, K, E, A, H, cap, **kw)


def ref(L):
    return C.byref(L) if L is not None else None


def norm(L, eps=1e-6, x=P, r=P, w=P, s=P, o=P, q=P, sc=P):
    return ep.lib.ep_rms_norm(ref(L), x, r, w, eps, s, o, q, sc, None)


def norm_bwd(L, eps=1e-6, g=P, gs=P, x=P, w=P, gx=P, gw=P, ws=P, nb=BIG):
    return ep.lib.ep_rms_norm_bwd(ref(L), g, gs, x, w, eps, gx, gw, ws, nb, None)


def act(L, h=P, nb=BIG, gu=P, q=P, sc=P):
    return ep.lib.ep_swiglu_scaled(ref(L), h, nb, gu, q, sc, None)


def linear(L, n=64, h=P, nb=BIG, x=P, xs=P, w=P, ws=P, o=P):
    return ep.lib.ep_grouped_linear_scaled(ref(L), h, nb, x, xs, w, ws, o, n, None)


def layer(L, n=64, idx=P, tw=P, x=P, gu=P, gs=P, dn=P, ds=P, o=P, ws=P, nb=BIG):
    return ep.lib.ep_expert_layer(ref(L), idx, tw, x, gu, gs, dn, ds, o, n, ws, nb, None)


def layer16(L, **kw):
    return layer(L, gs=None, ds=None, **kw)


ALL = [norm, norm_bwd, act, linear, layer, layer16]


@pytest.mark.parametrize("call", ALL)
def test_layout_checks(call):
    assert call(None) == ep.EP_ERR_NULL
    assert call(lay(K=0)) == ep.EP_ERR_SHAPE
    assert call(lay(H=12)) == ep.EP_ERR_SHAPE
    assert call(lay(cap=-1)) == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("call", [act, linear])
def test_handle_checks(call):
    L = lay()
    assert call(L, h=None) == ep.EP_ERR_NULL
    assert call(L, nb=ep.handle_regions(L).maps_bytes - 1) == ep.EP_ERR_HANDLE_SIZE
    assert call(L, h=MIS) == ep.EP_ERR_ALIGN


@pytest.mark.parametrize("call", [linear, layer, layer16])
@pytest.mark.parametrize("n", [-8, 0, 4, 12, (1 << 20) + 16, 1 << 40])
def test_feature_counts(call, n):
    assert call(lay(), n=n) == ep.EP_ERR_SHAPE
    assert call(lay(H=(1 << 20) + 64)) == ep.EP_ERR_SHAPE


def test_eight_bit_rows_are_whole_vectors():
    assert norm(lay(H=72)) == norm(lay(H=72), o=None) == ep.EP_ERR_SHAPE
    assert act(lay(H=72)) == linear(lay(H=72)) == layer(lay(H=72)) == ep.EP_ERR_SHAPE
    assert layer(lay(), n=72) == ep.EP_ERR_SHAPE
    # the 16-bit forms take any multiple of 8: the next check is what refuses
    assert norm(lay(H=72), q=None, sc=None, x=MIS) == ep.EP_ERR_ALIGN
    assert layer16(lay(H=72), n=72, x=MIS) == ep.EP_ERR_ALIGN
    assert linear(lay(), n=72, x=MIS) == ep.EP_ERR_ALIGN


def test_payload_types():
    for call in (linear, layer, layer16):
        assert call(lay(dtype="fp32")) == ep.EP_ERR_SHAPE
        assert call(lay(dtype="fp16"), x=MIS) == ep.EP_ERR_ALIGN
    for call in (norm, norm_bwd):
        assert call(lay(dtype="fp32"), x=MIS) == ep.EP_ERR_ALIGN
    assert act(lay(dtype="fp32"), gu=MIS) == ep.EP_ERR_ALIGN


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_sizes(call):
    assert call(lay(H=16384), x=MIS) == ep.EP_ERR_ALIGN
    assert call(lay(H=16400)) == ep.EP_ERR_SHAPE
    for eps in (-1e-6, float("nan")):
        assert call(lay(), eps=eps) == ep.EP_ERR_SHAPE
    assert call(lay(), eps=0.0, x=MIS) == ep.EP_ERR_ALIGN


def test_layer_routes():
    assert layer16(lay(T=512, K=2), x=MIS) == ep.EP_ERR_ALIGN
    assert layer16(lay(T=513, K=2)) == ep.EP_ERR_SHAPE
    assert layer16(lay(T=17, K=64, E=64)) == ep.EP_ERR_SHAPE


@pytest.mark.parametrize("call,names", [
    (norm, ("x", "w")), (norm_bwd, ("g", "x", "w", "gx", "ws")), (act, ("gu", "q", "sc")),
    (linear, ("x", "xs", "w", "ws", "o")),
    (layer, ("idx", "tw", "x", "gu", "gs", "dn", "ds", "o", "ws")),
    (layer16, ("idx", "tw", "x", "gu", "dn", "o", "ws"))])
def test_required_pointers_and_alignment(call, names):
    for name in names:
        assert call(lay(), **{name: None}) == ep.EP_ERR_NULL, name
        assert call(lay(), **{name: MIS}) == ep.EP_ERR_ALIGN, name


def test_pairs():
    L = lay()
    assert norm(L, o=None, q=None, sc=None) == ep.EP_ERR_NULL
    assert norm(L, q=None) == norm(L, sc=None) == ep.EP_ERR_NULL
    assert norm(L, r=None) == norm(L, s=None) == ep.EP_ERR_NULL
    for name in ("r", "s", "o", "q", "sc"):
        assert norm(L, **{name: MIS}) == ep.EP_ERR_ALIGN
    for name in ("gs", "gw"):
        assert norm_bwd(L, **{name: MIS}) == ep.EP_ERR_ALIGN
    assert layer(L, gs=None) == layer(L, ds=None) == ep.EP_ERR_NULL


def test_workspaces():
    L = lay()
    n = ep.lib.ep_rms_norm_bwd_workspace(C.byref(L))
    assert 0 < n <= 512 * L.H * 4
    assert norm_bwd(L, nb=n - 1) == ep.EP_ERR_WORKSPACE
    assert norm_bwd(L, nb=n, x=MIS) == ep.EP_ERR_ALIGN
    assert norm_bwd(L, gw=None, ws=None, nb=0, x=MIS) == ep.EP_ERR_ALIGN
    assert ep.lib.ep_rms_norm_bwd_workspace(C.byref(lay(T=1 << 20, H=16384))) <= 512 * 16384 * 4
    for bad in (lay(H=16400), lay(K=0), None):
        assert ep.lib.ep_rms_norm_bwd_workspace(ref(bad)) == 0
    n = ep.lib.ep_expert_layer_workspace(C.byref(L), 64)
    # the activations and products of every route
    assert n >= 16 * 2 * (64 * 2 + 64 * 4)
    assert layer(L, nb=n - 1) == layer16(L, nb=n - 1) == ep.EP_ERR_WORKSPACE
    assert layer(L, nb=n, x=MIS) == ep.EP_ERR_ALIGN
    for bad, inner in ((L, 0), (L, 12), (lay(T=513), 64), (lay(dtype="fp32"), 64), (None, 64)):
        assert ep.lib.ep_expert_layer_workspace(ref(bad), inner) == 0
    assert "workspace" in ep.status_str(ep.EP_ERR_WORKSPACE)


def test_no_tokens_is_no_work():
    # returns ahead of any HIP call: there is no device here
    L = lay(T=0)
    assert norm(L, x=None, r=None, s=None) == ep.EP_OK
    assert norm_bwd(L, g=None, x=None, gx=None, gs=None, gw=None, ws=None) == ep.EP_OK
    assert layer(L, idx=None, tw=None, x=None, o=None, ws=None, nb=0) == ep.EP_OK


def test_scale_columns():
    assert [ep.scale_columns(h) for h in (16, 128, 1024, 1040, 2048, 7168, 14336)] == \
        [8, 8, 8, 16, 16, 56, 112]


def test_binding_checks():
    L = lay()
    cpu = torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        ep.rms_norm(L, cpu, cpu[0], 1e-6, out=cpu)
    with pytest.raises(TypeError, match="x must be"):
        ep.rms_norm(L, cpu.float(), cpu[0], 1e-6, out=cpu)
    with pytest.raises(ValueError, match="down must have shape"):
        ep.expert_layer(L, cpu, cpu, cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="invalid layout"):
        ep.new_rms_norm_bwd_workspace(lay(H=16400))
    with pytest.raises(ValueError, match="invalid layout or inner"):
        ep.new_expert_layer_workspace(L, 12)


def test_eight_bit_weights_that_want_a_gradient():
    from combine_ep_prepare_amd import autograd as epa
    q, w = torch.zeros(4, 64, dtype=ep.E4M3), torch.zeros(1, 64, 64, dtype=ep.E4M3)
    s = torch.zeros(4, ep.scale_columns(64))
    with pytest.raises(RuntimeError, match="no backward"):
        epa.grouped_linear_scaled(q, s, w.requires_grad_(), s, None)
    with pytest.raises(RuntimeError, match="no backward"):
        epa.dispatch_scaled(q, s.clone().requires_grad_(), torch.zeros(4, 1), None)
