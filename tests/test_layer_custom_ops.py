"""The custom ops of the norm, the 8-bit ops and the layer for a few tokens: fake
shapes on the host; on the GPU the binding's own results, and gradients."""
import pytest
import torch

import combine_ep_prepare_amd as ep
import combine_ep_prepare_amd.custom_ops as co
from combine_ep_prepare_amd import autograd as epa

T, K, E, A, H, I = 24, 2, 4, 8, 144, 48
CAP = T * K + E * (A - 1)


def test_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    ll = co.layout_list(ep.Layout(T, K, E, A, 128, CAP, dtype="fp16"))
    with FakeTensorMode():
        h, x = torch.empty(8, dtype=torch.uint8), torch.empty(T, H, dtype=torch.float16)
        w = torch.empty(H, dtype=torch.float16)
        assert co.rms_norm(x, w, 1e-6).shape == (T, H)
        y, s = co.add_rms_norm(x, x, w, 1e-6)
        assert y.shape == s.shape == (T, H) and s.dtype == torch.float16
        gx, gw = co.rms_norm_bwd(x, x, w, 1e-6, None)
        assert gx.shape == (T, H) and gw.shape == (H,)
        assert co.rms_norm_grad_x(x, x, w, 1e-6, x).shape == (T, H)
        for q, scales, *more in (co.rms_norm_scaled(x, w, 1e-6),
                                 co.add_rms_norm_scaled(x, x, w, 1e-6)):
            assert q.shape == (T, H) and q.dtype == ep.E4M3
            assert scales.shape == (T, 8) and scales.dtype == torch.float32
            assert all(t.shape == (T, H) for t in more)
        q, scales = co.swiglu_scaled(torch.empty(CAP, 2 * I, dtype=torch.float16), h, ll)
        assert q.shape == (CAP, I) and scales.shape == (CAP, 8)
        w8 = torch.empty(E, H, I, dtype=ep.E4M3)
        out = co.grouped_linear_scaled(q, scales, w8, torch.empty(E, 2, 1), h, ll)
        assert out.shape == (CAP, H) and out.dtype == torch.float16
        idx = torch.empty(T, K, dtype=torch.int64)
        out = co.expert_layer(x, idx, torch.empty(T, K), torch.empty(E, 2 * I, H), w8, None, None)
        assert out.shape == (T, H) and out.dtype == torch.float16


@pytest.mark.parametrize("want", [(True, True, True), (True, False, False), (False, True, False),
                                  (False, False, True)])
def test_only_the_gradients_asked_for(monkeypatch, want):
    calls = []

    def forward(L, x, weight, eps, out=None, residual=None, sum_out=None, **kw):
        out.zero_()
        sum_out.zero_()

    def backward(L, grad, x, weight, eps, grad_x, grad_weight=None, workspace=None, grad_sum=None):
        calls.append(grad_weight is not None)
        assert (workspace is not None) == (grad_weight is not None)
        for t in (grad_x, grad_weight):
            if t is not None:
                t.fill_(1)

    monkeypatch.setattr(co, "_rms_norm", forward)
    monkeypatch.setattr(co, "_rms_norm_bwd", backward)
    monkeypatch.setattr(co, "new_rms_norm_bwd_workspace", lambda L, device: torch.empty(1))
    x, res, w = (torch.randn(*s, requires_grad=r) for s, r in zip(((T, H), (T, H), (H,)), want))
    y, s = co.add_rms_norm(x, res, w, 1e-6)
    (y.sum() + s.sum()).backward()
    assert calls == [want[2]]
    assert [t.grad is not None for t in (x, res, w)] == list(want)


@pytest.fixture
def gen():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.Generator(device="cuda").manual_seed(3)


def e4m3(gen, *shape):
    return (torch.randn(*shape, device="cuda", generator=gen) * 60).clamp(-448, 448).to(ep.E4M3)


@pytest.mark.gpu
def test_norm_and_its_gradients(gen):
    x, res, g, gs = (torch.randn(T, H, device="cuda", generator=gen).bfloat16() for _ in range(4))
    w = torch.randn(H, device="cuda", generator=gen).bfloat16()
    leaves = [t.clone().requires_grad_() for t in (x, res, w)]
    mine = [t.clone().requires_grad_() for t in (x, res, w)]
    y, s = co.add_rms_norm(*leaves, 1e-6)
    y2, s2 = epa.rms_norm(mine[0], mine[2], 1e-6, residual=mine[1])
    assert torch.equal(y, y2) and torch.equal(s, s2)
    torch.autograd.backward((y, s), (g, gs))
    torch.autograd.backward((y2, s2), (g, gs))
    for a, b in zip(leaves, mine):
        assert torch.equal(a.grad, b.grad)
    # without a residual, and one gradient alone: the same bits
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    co.rms_norm(a, w, 1e-6).backward(g)
    epa.rms_norm(b, w, 1e-6).backward(g)
    assert torch.equal(a.grad, b.grad)
    # only the sum is used: its gradient passes through
    c = x.clone().requires_grad_()
    epa.rms_norm(c, w, 1e-6, residual=res)[1].backward(gs)
    assert torch.equal(c.grad, gs)
    torch.library.opcheck(co.rms_norm, (x.clone().requires_grad_(), w, 1e-6))
    torch.library.opcheck(co.rms_norm_bwd, (g, x, w, 1e-6, gs))
    torch.library.opcheck(co.rms_norm_grad_x, (g, x, w, 1e-6, None))


@pytest.mark.gpu
def test_eight_bit_ops_and_layer(gen):
    def same(a, b):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))

    ll = co.layout_list(ep.Layout(T, K, E, A, H, CAP))
    idx = torch.randint(-1, E, (T, K), device="cuda", generator=gen)
    routing = epa.EpRouting(idx, E, A, H, CAP)
    x, res = (torch.randn(T, H, device="cuda", generator=gen).bfloat16() for _ in range(2))
    w = torch.ones(H, device="cuda").bfloat16()
    q, scales, total = epa.rms_norm_scaled(x, w, 1e-6, residual=res)
    same(co.add_rms_norm_scaled(x, res, w, 1e-6), (q, scales, total))
    same(co.rms_norm_scaled(total, w, 1e-6), (q, scales))
    tw = torch.rand(T, K, device="cuda", generator=gen)
    rq, rs, _ = epa.dispatch_scaled(q, scales, tw, routing)
    w1, w2 = e4m3(gen, E, 2 * I, H), e4m3(gen, E, H, I)
    s1, s2 = (torch.rand(E, *s, device="cuda", generator=gen) / 100 for s in ((1, 2), (2, 1)))
    gu = epa.grouped_linear_scaled(rq, rs, w1, s1, routing)
    same([co.grouped_linear_scaled(rq, rs, w1, s1, routing.handle, ll)], [gu])
    same(co.swiglu_scaled(gu, routing.handle, ll), epa.swiglu_scaled(gu, routing))
    same([co.expert_layer(x, idx, tw, w1, w2, s1, s2)],
         [epa.expert_layer(x, idx, tw, w1, w2, s1, s2)])
    # the schema's check multiplies tensors, which torch does not do in 8 bits
    utils = ("test_autograd_registration", "test_faketensor")
    torch.library.opcheck(co.swiglu_scaled, (gu, routing.handle, ll), test_utils=utils)
    torch.library.opcheck(co.expert_layer, (x, idx, tw, w1, w2, s1, s2), test_utils=utils)


@pytest.mark.gpu
def test_dispatch_in_eight_bits_copies(gen):
    """Rows and scales arrive bit for bit, NaN patterns too; pads and tail are zeros."""
    idx = torch.randint(-1, E, (T, K), device="cuda", generator=gen)
    routing = epa.EpRouting(idx, E, A, 1040)
    q = torch.randint(0, 256, (T, 1040), device="cuda", generator=gen, dtype=torch.uint8)
    scales = torch.rand(T, 16, device="cuda", generator=gen)
    scales[3, 2] = float("nan")
    rq, rs, rw = epa.dispatch_scaled(q.view(ep.E4M3), scales, torch.rand(T, K, device="cuda"),
                                     routing)
    maps = ep.handle_maps(routing.layout, routing.handle)
    total = int(routing.expert_offsets[-1])
    src = torch.full((rq.shape[0],), -1, device="cuda")
    src[:total] = maps["row_src"][:total].long()
    live = src >= 0
    assert torch.equal(rq.view(torch.uint8)[live], q[src[live] // K])
    assert torch.equal(rs.view(torch.int32)[live], scales.view(torch.int32)[src[live] // K])
    assert not rq.view(torch.uint8)[~live].any() and not rs[~live].any()
    with pytest.raises(ValueError, match="not rows in 8 bits"):
        epa.dispatch_scaled(q, scales, torch.rand(T, K, device="cuda"), routing)
    with pytest.raises(ValueError, match="not rows in 8 bits"):
        epa.dispatch_scaled(q.view(ep.E4M3), scales[:, :8], torch.rand(T, K, device="cuda"), routing)
