"""The grouped linear's custom op computes the gradients that are asked for and
no other: on the host with the binding's calls stood in for, and on the GPU."""
import pytest
import torch

import combine_ep_prepare_amd as ep
import combine_ep_prepare_amd.custom_ops as co

WANTED = [(True, True), (True, False), (False, True)]
T, K, E, A, H, N = 48, 2, 4, 8, 64, 72
CAP = T * K + E * (A - 1)


@pytest.mark.parametrize("want_x,want_w", WANTED)
def test_only_the_gradients_asked_for(monkeypatch, want_x, want_w):
    calls = []

    def forward(L, handle, x, weight, out, stream=None):
        out.zero_()

    def backward(L, handle, grad, x, weight, grad_x=None, grad_weight=None, stream=None):
        calls.append((grad_x is not None, grad_weight is not None))
        assert (weight is not None) >= want_x and (x is not None) >= want_w
        for t, shape in ((grad_x, (CAP, H)), (grad_weight, (E, N, H))):
            if t is not None:
                assert t.shape == shape
                t.fill_(1)

    monkeypatch.setattr(co, "_grouped_linear", forward)
    monkeypatch.setattr(co, "_grouped_linear_bwd", backward)
    ll = co.layout_list(ep.Layout(T, K, E, A, 128, CAP, dtype="fp32"))
    x = torch.randn(CAP, H, requires_grad=want_x)
    w = torch.randn(E, N, H, requires_grad=want_w)
    co.grouped_linear(x, w, torch.empty(8, dtype=torch.uint8), ll).sum().backward()
    assert calls == [(want_x, want_w)]
    assert (x.grad is not None) == want_x and (w.grad is not None) == want_w


def test_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    ll = co.layout_list(ep.Layout(T, K, E, A, 128, CAP, dtype="fp16"))
    with FakeTensorMode():
        h = torch.empty(8, dtype=torch.uint8)
        g = torch.empty(CAP, N, dtype=torch.float16)
        gx = co.grouped_linear_grad_x(g, torch.empty(E, N, H, dtype=torch.float16), h, ll)
        gw = co.grouped_linear_grad_weight(g, torch.empty(CAP, H, dtype=torch.float16), h, ll)
    assert gx.shape == (CAP, H) and gw.shape == (E, N, H)
    assert gx.dtype == gw.dtype == torch.float16


@pytest.mark.gpu
@pytest.mark.parametrize("want_x,want_w", WANTED)
def test_one_gradient_has_the_bits_of_both(want_x, want_w):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(5)
    ll = co.layout_list(ep.Layout(T, K, E, A, H, CAP))
    handle = torch.empty(ep.handle_mem_size(ep.Layout(T, K, E, A, H, CAP)), dtype=torch.uint8,
                         device="cuda")
    co.prepare(torch.randint(0, E, (T, K), device="cuda", generator=gen), handle, ll)
    x, w, g = (torch.randn(*s, device="cuda", generator=gen).bfloat16()
               for s in ((CAP, H), (E, N, H), (CAP, N)))
    gx, gw = co.grouped_linear_bwd(g, x, w, handle, ll)
    x.requires_grad_(want_x)
    w.requires_grad_(want_w)
    co.grouped_linear(x, w, handle, ll).backward(g)
    for t, want, whole in ((x, want_x, gx), (w, want_w, gw)):
        assert torch.equal(t.grad, whole) if want else t.grad is None
    torch.library.opcheck(co.grouped_linear_grad_x, (g, w.detach(), handle, ll))
    torch.library.opcheck(co.grouped_linear_grad_weight, (g, x.detach(), handle, ll))
