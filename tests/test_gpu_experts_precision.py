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
