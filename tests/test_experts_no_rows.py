"""The grouped linear's backward where the buffers hold no row: an empty tensor's
pointer is NULL, and asking for grad_x alone is a call like any other."""
import ctypes as C

import pytest
import torch

import combine_ep_prepare_amd as ep

P = C.c_void_p(0x10000)            # fake, never dereferenced
MIS = C.c_void_p(0x10008)


def call(L, gx, gw, weight=P, grad=P):
    return ep.lib.ep_grouped_linear_bwd(C.byref(L), P, 1 << 30, grad, P, weight, gx, gw, 64, None)


def test_no_output_is_needed_where_there_is_no_row():
    L = ep.Layout(16, 2, 4, 8, 64, 0)
    assert call(L, None, None, grad=MIS) == ep.EP_ERR_ALIGN        # past the NULL checks
    assert call(L, None, P, weight=None, grad=MIS) == ep.EP_ERR_ALIGN
    assert call(ep.Layout(16, 2, 4, 8, 64, 96), None, None, grad=MIS) == ep.EP_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("want", ["x", "w", "both"])
def test_empty_buffers(dtype, want):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    E, H, N = 4, 64, 72
    L = ep.Layout(16, 2, E, 8, H, 0, dtype=dtype)
    handle = ep.new_handle(L)
    ep.prepare(L, torch.zeros(16, 2, dtype=torch.int64, device="cuda"),
               torch.empty(E, dtype=torch.int32, device="cuda"), handle)
    x, g = (torch.empty(0, n, dtype=dtype, device="cuda") for n in (H, N))
    w = torch.ones(E, N, H, dtype=dtype, device="cuda")
    gx = torch.empty_like(x) if want != "w" else None
    gw = torch.full_like(w, 5) if want != "x" else None
    ep.grouped_linear_bwd(L, handle, g, x, w, gx, gw)
    assert gw is None or not gw.any()
    torch.cuda.synchronize()
