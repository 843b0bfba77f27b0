"""How many bits the experts' activation and 4-bit product keep.

Inputs on which a lossy intermediate shows in the result: gates far from zero,
weights that mostly equal their zero point, rows with a mean. Tolerances are
bounds, not measurements: a unit below is half a step of fp32, 2^-24 relative.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_experts import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def activation(c, gate, up, grad):
    """swiglu and its gradient of rows [T,H], every row live."""
    T, H = gate.shape
    L = c.layout(H)
    gu = torch.cat((gate, up), 1).cuda()
    out, dgu = c.out(T, H), c.out(T, 2 * H)
    ep.swiglu(L, c.handle, gu, out)
    ep.swiglu_bwd(L, c.handle, grad.cuda(), gu, dgu)
    return [t.double().cpu() for t in (out, dgu[:, :H], dgu[:, H:])]


def activation64(gate, up, grad):
    """The definition, and the magnitudes that 1 + g (1 - s) adds up."""
    g, u, d = gate.double(), up.double(), grad.double()
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    wants = (g * s * u, d * u * (s * (1 + g * rest)), d * g * s)
    return wants, (wants[0].abs(), (d * u).abs() * s * (1 + (g * rest).abs()), wants[2].abs())


def rows(seed, T, H, low, high, up_scale, dtype):
    gen = torch.Generator().manual_seed(seed)
    gate = (torch.rand(T, H, generator=gen) * (high - low) + low).to(dtype)
    up = (torch.randn(T, H, generator=gen) * up_scale).to(dtype)
    return gate, up, torch.randn(T, H, generator=gen).to(dtype)


# exp(-|g|) as a square: the root within 4 units (the hardware's exp2 2, its
# correction 2), twice in the square and once more for its rounding, 9. 1 + e and
# the reciprocal: e's error counts at most half in 1 / (1 + e), 4.5, and their
# own two roundings 3. The results multiply two roots, the reciprocal and the
# inputs: 8 + 7.5 and at most five roundings; 1 + g q adds q's error (its e and r,
# and a rounding) to the terms it sums: 18 more and two roundings.
UNITS = 22, 42, 22


@pytest.mark.parametrize("low,high,up_scale", [(-4, 4, 1.0), (-30, 30, 1.0), (-87, 88, 1.0),
                                               (-87, -60, 1.0), (-170, -80, 2.0 ** 100),
                                               (-2, -1, 1.0)])
def test_fp32_activation_at_full_precision(low, high, up_scale):
    T, H = 64, 1024
    c = Case("one", T, 1, 2, 1, "fp32", cap=T)
    args = rows(7, T, H, low, high, up_scale, torch.float32)
    wants, mags = activation64(*args)
    for name, got, want, mag, units in zip(("out", "d_gate", "d_up"), activation(c, *args),
                                           wants, mags, UNITS):
        # results below the smallest normal number keep its step, 2^-149; a factor
        # that is subnormal on the way stands beside one below 2^7 (|g|, 1 + |g|,
        # or the gradient)
        over = (got - want).abs() - units * 2.0 ** -24 * mag - 2.0 ** -141
        assert over.max() <= 0, (name, int((over > 0).sum()), float(over.max()))


@pytest.mark.parametrize("up_scale", [1.0, 2.0 ** 40])
def test_bf16_activation_of_gates_below_minus_87(up_scale):
    """bf16 has fp32's range: silu(-88) is a normal number, and so is what a
    sigmoid below that range gives with a large factor."""
    T, H = 64, 256
    c = Case("one", T, 1, 2, 1, "bf16", cap=T)
    args = rows(8, T, H, -110, -80, up_scale, torch.bfloat16)
    wants, mags = activation64(*args)
    for name, got, want, mag in zip(("out", "d_gate", "d_up"), activation(c, *args), wants, mags):
        # the exponent's rounding, |g| and a quarter units (log2(e) in fp32), besides
        # the units above; then the rounding to bf16, of subnormals 2^-134
        rel = (42 + 1.25 * 110) * 2.0 ** -24
        tol = rel * mag + 2.0 ** -8 * want.abs() * (1 + rel) + 2.0 ** -133
        over = (got - want).abs() - tol
        assert over.max() <= 0, (name, int((over > 0).sum()), float(over.max()))
        if name != "d_up" and up_scale > 1:
            assert (got != 0).float().mean() > 0.9


# --------------------------------------------------------------------------
# 4-bit weights
# --------------------------------------------------------------------------

def packed(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def quant(c, x, q, scales, zeros):
    E, N, H = q.shape
    out = c.out(c.cap, N)
    ep.grouped_linear_quant(c.layout(H), c.handle, x.cuda(), packed(q).cuda(), scales.cuda(),
                            None if zeros is None else zeros.cuda(), out)
    return out.double().cpu()


def quant64(c, x, q, scales, zeros, G):
    """The definition, and the magnitudes (q - z) x s that it adds up."""
    E, N, H = q.shape
    z = torch.full(scales.shape, 8.0) if zeros is None else zeros
    w = (q.double().reshape(E, N, -1, G) - z.double()[..., None]) * scales.double()[..., None]
    w = w.reshape(E, N, H)
    want, mags = (torch.zeros(c.cap, N, dtype=torch.float64) for _ in range(2))
    for e, (a, b) in enumerate(c.rows):
        want[a:b] = x[a:b].double() @ w[e].t()
        mags[a:b] = x[a:b].double().abs() @ w[e].abs().t()
    return want, mags


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_4_bit_weights_near_their_zero_point(dtype, G, zeros):
    """One weight in sixteen differs from its zero point, by one, and x is
    positive: the sums of q x and of z x are hundreds of times the result."""
    T, E, N, H = 19, 2, 72, 640
    c = Case("one", T, 1, E, 1, dtype)
    g = c.gen
    # 8 bits over four powers of two, steps of 2^-7; the inputs that count in [1, 2)
    x = (1 + torch.randint(0, 128, (c.cap, H), generator=g) / 128) * \
        2.0 ** torch.randint(0, 4, (c.cap, H), generator=g)
    x[:, ::16] = 1 + torch.randint(0, 128, (c.cap, H // 16), generator=g) / 128
    x = x.to(c.dtype)
    x[~c.live] = float("nan")
    z = torch.randint(1, 15, (E, N, H // G), generator=g, dtype=torch.uint8) if zeros else None
    q = torch.full((E, N, H), 8, dtype=torch.uint8) if z is None else \
        z.repeat_interleave(G, 2).clone()
    q[..., ::16] += torch.randint(0, 3, (E, N, H // 16), generator=g, dtype=torch.uint8) - 1
    s = (torch.rand(E, N, H // G, generator=g) * 0.01 + 1e-3).to(c.dtype)
    got = quant(c, x, q, s, z)
    want, mags = quant64(c, x, q, s, z, G)
    # a group's sums are exact: of whole multiples of 2^-7, up to 31 * 16 * 128 =
    # 2^15.9 in size, 23 bits. The scales and the sum over groups and wavefronts
    # round: at most two steps a group and eight more.
    bound = (2 * (H // G) + 8) * 2.0 ** -23 * mags
    tol = bound + c.eps2 * (want.abs() + bound) + c.tiny
    over = ((got - want).abs() - tol)[c.live]
    assert over.max() <= 0, (int((over > 0).sum()), float(over.max()))


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [3, 700])
def test_4_bit_zero_points_of_any_byte(T, dtype, G):
    """Zero points from 0 to 255, and rows with a mean; few rows an expert and
    many."""
    E, N, H = 3, 136, 384
    c = Case("steep", T, 1, E, 4, dtype, zero_tail=True)
    x = c.buffer(H) + 2
    q = torch.randint(0, 16, (E, N, H), generator=c.gen, dtype=torch.uint8)
    z = torch.randint(0, 256, (E, N, H // G), generator=c.gen, dtype=torch.uint8)
    z[0, 0], z[0, 1] = 0, 255
    s = (torch.rand(E, N, H // G, generator=c.gen) * 1e-3 + 1e-4).to(c.dtype)
    got = quant(c, x, q, s, z)
    want, mags = quant64(c, x, q, s, z, G)
    # fp16: the definition's own sums; bf16: those of (16 + q) x and (16 + z) x
    bound = (H + 8) * 2.0 ** -23 * mags
    if dtype == "bf16":
        for e, (a, b) in enumerate(c.rows):
            terms = (32.0 + 15 + z[e].double()) * s[e].double()
            bound[a:b] += (G + 8) * 2.0 ** -23 * (x[a:b].double().abs()
                                                  @ terms.repeat_interleave(G, 1).t())
    tol = bound + c.eps2 * (want.abs() + bound) + c.tiny
    over = ((got - want).abs() - tol)[c.live]
    assert over.max() <= 0, (int((over > 0).sum()), float(over.max()))


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 65504.0])
@pytest.mark.parametrize("zeros", [False, True])
def test_4_bit_fp16_special_values_follow_the_definition(value, zeros):
    T, E, N, H, G = 21, 2, 40, 256, 64
    c = Case("one", T, 1, E, 1, "fp16")
    x = c.buffer(H)
    q = torch.randint(0, 16, (E, N, H), generator=c.gen, dtype=torch.uint8)
    z = torch.randint(0, 16, (E, N, H // G), generator=c.gen, dtype=torch.uint8) if zeros else None
    s = torch.full((E, N, H // G), 0.5 ** 10, dtype=torch.float16)
    r = c.rows[E - 1][0] + 5
    x[r, 70] = value
    got = quant(c, x, q, s, z)
    want, _ = quant64(c, x, q, s, z, G)
    assert torch.equal(got[c.live].isnan(), want[c.live].isnan())
    assert torch.equal(got[c.live].isinf(), want[c.live].isinf())
    inf = want.isinf() & c.live[:, None]
    assert torch.equal(got[inf], want[inf])
