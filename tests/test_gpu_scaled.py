"""The experts' product and activation in 8 bits against 64-bit references.

Pad and tail rows of every input hold NaN, of values and of scales, and outputs are
pre-filled, as in test_gpu_experts. Tolerances are bounds:

- the 8-bit matrix instruction takes eight neighbouring products of k at a time. It
  aligns them to the exponent of the largest (the sum of its factors' exponents, so
  at most its magnitude) and cuts each off 13 bits below: beside a product of 2^16
  one of 2^3 counts and one of 2^2 does not, where eight places on 2^-7 still
  counts. Each of the eight loses less than 2^-13 of the largest, the group less
  than 2^-10 of it; and the largest product is at most the product of the largest
  factors. Values that are small whole numbers lose nothing;
- the groups' sums, n of them, held in fp32, are off by at most n steps of 2^-23 of
  the sum of the terms' magnitudes; each block's sum then takes a product of scales
  and a fused multiply-add: 4 steps more a block;
- one rounding to the payload type at the end: half a step;
- the activation's values are within 24 u of their magnitude in fp32 (u = 2^-24:
  exp2 and the reciprocal within a unit each, a gate of up to 8 takes the exponent
  off by 4 u, half a dozen products), and in 8 bits off by half a step of e4m3.
"""
import numpy as np
import pytest
import torch

import combine_ep_prepare_amd as ep
from combine_ep_prepare_amd import autograd as epa
from test_gpu_experts import CANARY, DT, SHAPES, Case, sum_bound
from test_gpu_norm import U, check_scaled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def to_e4m3(t):
    return t.clamp(-448, 448).to(ep.E4M3)


def weights(gen, E, N, H):
    """e4m3 weights [E,N,H] and scales of every size, and what they stand for in fp64."""
    q = to_e4m3(torch.randn(E, N, H, generator=gen) * 90)
    nb, kb = -(-N // 128), -(-H // 128)
    s = torch.exp2(torch.randn(E, nb, kb, generator=gen) - 7) * H ** -0.5
    wide = s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :H]
    return q, s, q.double() * wide


def rows8(gen, cap, H, live):
    """e4m3 rows [cap,H] with scales, NaN where no route is, and their values in fp64."""
    q = torch.randn(cap, H, generator=gen) * 90
    s = torch.exp2(torch.randn(cap, ep.scale_columns(H), generator=gen) - 6)
    q[~live] = float("nan")
    q = to_e4m3(q)
    s[~live] = float("nan")
    s[:, -(-H // 128):] = float("nan")      # columns past the blocks are not read
    wide = s.double().repeat_interleave(128, 1)[:, :H]
    return q, s, q.double() * wide


def largest(v):
    """The largest magnitude of each eight of a row."""
    return torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2)


def linear_case(c, H, N, whole=False):
    """With `whole`, values are small whole numbers and scales powers of two near
    each other: every sum is exact in fp32, and only the last rounding is left."""
    L = c.layout(H)
    if whole:
        x = torch.randint(-15, 16, (c.cap, H), generator=c.gen).float()
        w = torch.randint(-15, 16, (c.E, N, H), generator=c.gen).float()
        xs = torch.exp2(torch.randint(-2, 3, (c.cap, ep.scale_columns(H)), generator=c.gen))
        ws = torch.exp2(torch.randint(-2, 3, (c.E, -(-N // 128), -(-H // 128)), generator=c.gen) - 9)
        xv = x.double() * xs.double().repeat_interleave(128, 1)[:, :H]
        wv = w.double() * ws.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :H]
        x, w = to_e4m3(x), to_e4m3(w)
    else:
        x, xs, xv = rows8(c.gen, c.cap, H, c.live)
        w, ws, wv = weights(c.gen, c.E, N, H)
    out = c.out(c.cap, N)
    ep.grouped_linear_scaled(L, c.handle, x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out)
    want, mag = torch.zeros(c.cap, N, dtype=torch.float64), torch.zeros(c.cap, N, dtype=torch.float64)
    for e, (a, b) in enumerate(c.rows):
        want[a:b] = xv[a:b] @ wv[e].t()
        mag[a:b] = (sum_bound(H + 4 * (-(-H // 128)), xv[a:b].abs() @ wv[e].abs().t())
                    + 2.0 ** -10 * (largest(xv[a:b]) @ largest(wv[e]).t()))
    c.check_rows(out, want, torch.zeros_like(mag) if whole else mag, f"H={H} N={N}")
    return out


def round16(n):
    return -(-n // 16) * 16


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind,T,K,E,A,H,N", SHAPES)
def test_linear(kind, T, K, E, A, H, N, dtype):
    linear_case(Case(kind, T, K, E, A, dtype, seed=T + N), round16(H), N)


@pytest.mark.parametrize("kind,T,K,E,A,H,N", SHAPES)
def test_linear_of_whole_numbers(kind, T, K, E, A, H, N):
    """Sums below 225 * 16 * H * 2^-9, multiples of 2^-13: 24 bits hold them up to
    H = 1040 and more."""
    linear_case(Case(kind, T, K, E, A, "fp16", seed=T + N), round16(H), N, whole=True)


@pytest.mark.parametrize("fill_pads", [False, True])
@pytest.mark.parametrize("zero_tail", [False, True])
def test_linear_pads_and_capacity(fill_pads, zero_tail):
    """Both row policies, with a capacity that ends inside a segment."""
    c = Case("any", 60, 3, 7, 16, "bf16", seed=4, cap=150, fill_pads=fill_pads,
             zero_tail=zero_tail)
    linear_case(c, 272, 136)


@pytest.mark.parametrize("T,K,E,H,N", [
    (1, 1, 1, 16, 8), (1, 8, 8, 128, 128), (2, 2, 3, 112, 120), (16, 1, 1, 144, 136),
    (17, 1, 1, 384, 64), (129, 1, 1, 1152, 136), (300, 2, 2, 2064, 264), (1000, 1, 1, 640, 1032)])
def test_linear_edges(T, K, E, H, N):
    """Depths around a block and a step, features around a tile."""
    linear_case(Case("any", T, K, E, 1, "bf16", seed=T), H, N)
    linear_case(Case("any", T, K, E, 1, "bf16", seed=T), H, N, whole=True)


def test_linear_special_values():
    """A NaN value, an infinite or NaN scale reach their own outputs alone."""
    c = Case("any", 40, 2, 3, 4, "bf16", seed=9)
    H, N = 272, 264
    x, xs, _ = rows8(c.gen, c.cap, H, c.live)
    w, ws, _ = weights(c.gen, 3, N, H)
    (a, b), (a1, _) = c.rows[0], c.rows[1]
    assert b - a > 3
    x.view(torch.uint8)[a, 5] = 0x7F
    xs[a + 1, 2] = float("inf")
    xs[a1, 0] = float("nan")
    w.view(torch.uint8)[2, 7, 3] = 0xFF
    ws[1, 1, 1] = float("inf")
    out = c.out(c.cap, N)
    ep.grouped_linear_scaled(c.layout(H), c.handle, x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out)
    out = out.cpu()
    bad = torch.zeros(c.cap, N, dtype=torch.bool)
    bad[a] = bad[a + 1] = bad[a1] = True
    bad[c.rows[1][0]:c.rows[1][1], 128:256] = True
    bad[c.rows[2][0]:c.rows[2][1], 7] = True
    assert (out.isfinite() == ~bad)[c.live].all()


def act_case(c, inner, scale=1.0):
    L = c.layout(inner)
    gu = c.buffer(2 * inner, scale)
    q = torch.full((c.cap, inner), 7.0, device="cuda").to(ep.E4M3)
    s = torch.full((c.cap, ep.scale_columns(inner)), 7.0, device="cuda")
    ep.swiglu_scaled(L, c.handle, gu.cuda(), q, s)
    q, s = q.cpu(), s.cpu()
    g, u = gu.double().chunk(2, 1)
    check_scaled(q[c.live], s[c.live], (g * torch.sigmoid(g) * u)[c.live], 24 * U)
    dead = ~c.live
    for t, filler in ((q.float(), dead[:c.total].clone()), (s, dead[:c.total].clone())):
        assert (t[:c.total][filler] == (0.0 if c.flags["fill_pads"] else 7.0)).all()
        assert (t[c.total:] == (0.0 if c.flags["zero_tail"] else 7.0)).all()
    return q, s


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind,T,K,E,A,inner", [
    ("any", 0, 2, 3, 8, 64), ("none", 40, 2, 3, 8, 80), ("any", 1, 1, 1, 1, 16),
    ("masked", 7, 3, 16, 1, 128), ("any", 33, 4, 6, 16, 144), ("steep", 90, 2, 9, 1, 1040),
    ("one", 257, 1, 3, 128, 768), ("any", 700, 2, 5, 16, 2048), ("any", 20, 2, 3, 4, 14336)])
def test_activation(kind, T, K, E, A, inner, dtype):
    act_case(Case(kind, T, K, E, A, dtype, seed=T + inner), inner)


@pytest.mark.parametrize("fill_pads", [False, True])
@pytest.mark.parametrize("zero_tail", [False, True])
def test_activation_pads_and_capacity(fill_pads, zero_tail):
    act_case(Case("any", 60, 3, 7, 16, "fp16", seed=4, cap=150, fill_pads=fill_pads,
                  zero_tail=zero_tail), 272)


def test_refused_handle_writes_nothing():
    c = Case("any", 40, 2, 3, 8, "bf16")
    other = ep.Layout(41, 2, 3, 8, 64, c.cap)
    out = c.out(c.cap, 64)
    q, s = torch.zeros(c.cap, 64, device="cuda").to(ep.E4M3), torch.ones(c.cap, 8, device="cuda")
    w, ws = torch.zeros(3, 64, 64, device="cuda").to(ep.E4M3), torch.ones(3, 1, 1, device="cuda")
    ep.grouped_linear_scaled(other, c.handle, q, s, w, ws, out)
    assert (out == CANARY).all() and ep.read_status(c.handle) == ep.STATUS_LAYOUT
    c = Case("any", 40, 2, 3, 8, "bf16")
    ep.swiglu_scaled(other, c.handle, torch.ones(c.cap, 128, dtype=torch.bfloat16, device="cuda"), q, s)
    assert (q.float() == 0).all() and (s == 1).all()
    assert ep.read_status(c.handle) == ep.STATUS_LAYOUT


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,E,A,H,inner", [(40, 3, 6, 8, 272, 144), (5, 2, 9, 1, 1040, 528),
                                             (600, 2, 4, 16, 512, 256)])
def test_whole_layer(T, K, E, A, H, inner, dtype):
    """Norm, dispatch, product, activation, product and combine in 8 bits, each step
    checked from what it was given; eager, and captured and replayed."""
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(T)
    x, res = ((torch.randn(T, H, generator=gen)).to(dt).cuda() for _ in range(2))
    nw = torch.ones(H, dtype=dt, device="cuda")
    idx = torch.from_numpy(np.argsort(np.random.default_rng(T).random((T, E)), 1)[:, :K].copy()).cuda()
    idx[T // 2, 0] = -1
    tw = torch.rand(T, K, generator=gen).cuda()
    (w1, s1, v1), (w2, s2, v2) = weights(gen, E, 2 * inner, H), weights(gen, E, H, inner)
    w1, s1, w2, s2 = (t.cuda() for t in (w1, s1, w2, s2))

    def forward():
        q, sc, total = epa.rms_norm_scaled(x, nw, 1e-6, residual=res)
        routing = epa.EpRouting(idx, E, A, H)
        rq, rs, rw = epa.dispatch_scaled(q, sc, tw, routing)
        gu = epa.grouped_linear_scaled(rq, rs, w1, s1, routing, dt)
        aq, asc = epa.swiglu_scaled(gu, routing)
        y = epa.grouped_linear_scaled(aq, asc, w2, s2, routing, dt)
        return epa.combine(y, routing, rw), q, sc, total

    out, q, sc, total = forward()
    xv = q.double().cpu() * sc.double().cpu().repeat_interleave(128, 1)[:, :H]
    of = total.double().cpu()
    y = of / ((of ** 2).mean(1, keepdim=True) + 1e-6).sqrt()
    assert (xv - y).norm() <= 2 ** -4 * y.norm()
    want = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, k = (idx.cpu() == e).nonzero(as_tuple=True)
        g, u = (xv[t] @ v1[e].t()).chunk(2, 1)
        want.index_add_(0, t, tw.cpu()[t, k].double()[:, None] * ((g * torch.sigmoid(g) * u) @ v2[e].t()))
    # the activation's rounding to 8 bits: half a step, 2^-4 of each value at most,
    # and a norm of it on the sums, which the products' roundings do not reach
    assert (out.double().cpu() - want).norm() <= (2 ** -4 + 2 ** -6) * want.norm()

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        forward()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = forward()
    for _ in range(3):
        for t in again:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(again, (out, q, sc, total)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_gradients_are_refused():
    routing = epa.EpRouting(torch.zeros(4, 1, dtype=torch.int64, device="cuda"), 1, 1, 64)
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    gu = torch.randn(4, 128, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no backward"):
        epa.rms_norm_scaled(x, w, 1e-6)
    with pytest.raises(RuntimeError, match="no backward"):
        epa.swiglu_scaled(gu, routing)
    with torch.no_grad():
        epa.rms_norm_scaled(x, w, 1e-6)
        epa.swiglu_scaled(gu, routing)
    y = epa.rms_norm(x, w, 1e-6)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(y.sum(), x, create_graph=True)


@pytest.mark.parametrize("kind,T,K,E,A,H,N", [
    ("any", 140, 2, 40, 1, 528, 520), ("steep", 900, 2, 16, 4, 272, 1160),   # 64 x 64 tiles
    ("any", 1200, 2, 64, 1, 272, 1032), ("steep", 1200, 2, 64, 1, 272, 1032),   # 64 x 128
    ("masked", 1500, 4, 64, 8, 656, 1048), ("any", 960, 1, 8, 1, 400, 4104),   # 128 x 128
    ("steep", 1000, 1, 8, 2, 272, 4104),
    ("any", 6000, 2, 96, 1, 272, 1032), ("steep", 9000, 2, 64, 4, 400, 1288),   # 256 x 256
    ("any", 3300, 2, 8, 16, 144, 4104), ("one", 700, 1, 2, 1, 272, 16392),
    ("any", 1700, 2, 64, 1, 4112, 1032)])
def test_linear_tiles(kind, T, K, E, A, H, N):
    """Every tile size, of whole numbers: ragged rows, features, segments and last
    blocks, tiles with part of their rows, experts without any."""
    linear_case(Case(kind, T, K, E, A, "bf16", seed=T), H, N, whole=True)


@pytest.mark.parametrize("T,H,N", [(16400, 144, 136), (216000, 16, 264)])
def test_linear_many_experts(T, H, N):
    """The most experts, with a few rows each and with many: the longest tile lists."""
    linear_case(Case("any", T, 1, 2048, 1, "bf16", seed=1), H, N, whole=True)
