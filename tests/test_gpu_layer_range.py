"""The layer for a few tokens in fp16 where activations leave fp16's range, or lie so
low in it that its subnormals would take their last bits.

Gates are 30 and more, where silu(g) is g to fp32's last bit (exp(-30) < 2^-43), x
and the weights whole numbers times a power of two of few bits: both products' sums are
exact in fp32 in any order, activations take 22 bits at most, and what is left is the
result's own rounding, half a step. Where a step of the second product (64 values of k,
128 with 8-bit weights) holds activations of very different sizes, each may be off by
2^-36 of the largest.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_layer import Layer

pytestmark = pytest.mark.gpu

HALF = torch.finfo(torch.float16).eps / 2
TINY = torch.finfo(torch.float16).smallest_normal * HALF


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def whole(gen, top, *shape):
    """Whole numbers of e4m3: -top to top, top 15 at most."""
    return torch.randint(-top, top + 1, shape, generator=gen).double()


class Exact:
    """One expert of I = 256 features that every token goes to with weight 1. The first
    input is 1 and makes the gate, the others make up: gate [I], up [I, H - 1], down [H, I]
    are e4m3 values, each matrix times a power of two of its own."""

    def __init__(self, x, gate, up, down, up_power=0, down_power=0, x_power=0):
        T, I, H = x.shape[0], up.shape[0], up.shape[1] + 1
        self.x = torch.cat([torch.ones(T, 1).double(), x * 2.0 ** x_power], 1)
        self.gate = torch.cat([gate[:, None], torch.zeros(I, H - 1).double()], 1)
        self.up = torch.cat([torch.zeros(I, 1).double(), up], 1)
        self.down, self.powers = down, (2.0 ** up_power, 2.0 ** down_power)
        self.layout = ep.Layout(T, 1, 1, 1, H, 0, dtype=torch.float16)
        self.I = I

    def run(self, eight):
        up, down = self.powers
        x = self.x.half().cuda()
        assert (x.double().cpu() == self.x).all()
        scales = (None, None)
        if eight:
            w1 = torch.cat([self.gate, self.up])[None].float().to(ep.E4M3).cuda()
            w2 = self.down[None].float().to(ep.E4M3).cuda()
            blocks = self.I // 128
            s1 = torch.tensor([1.0] * blocks + [up] * blocks).reshape(1, -1, 1)
            scales = (s1.repeat(1, 1, -(-w1.shape[2] // 128)).contiguous().cuda(),
                      torch.full((1, -(-w2.shape[1] // 128), blocks), down).cuda())
            assert (w1.double().cpu()[0] == torch.cat([self.gate, self.up])).all()
        else:
            w1 = torch.cat([self.gate, self.up * up])[None].half().cuda()
            w2 = (self.down * down)[None].half().cuda()
            assert (w1.double().cpu()[0] == torch.cat([self.gate, self.up * up])).all()
            assert (w2.double().cpu()[0] == self.down * down).all()
        out = torch.full_like(x, 7.0)
        T = x.shape[0]
        ep.expert_layer(self.layout, torch.zeros(T, 1, dtype=torch.int64, device="cuda"),
                        torch.ones(T, 1, device="cuda"), x, w1, w2, out,
                        ep.new_expert_layer_workspace(self.layout, self.I).fill_(255), *scales)
        return out.double().cpu()

    def activations(self):
        return (self.x @ self.gate.t()) * (self.x @ self.up.t()) * self.powers[0]

    def check(self, eight, off=0.0):
        a = self.activations()
        want = a @ self.down.t() * self.powers[1]
        out = self.run(eight)
        bound = off + HALF * (want.abs() + off) + TINY
        assert out.isfinite().all() and ((out - want).abs() <= bound).all(), \
            float(((out - want).abs() - bound).max())


def few(gen, H, I, n):
    """[H, I] of -1 and 1 in n places of each row, zeros elsewhere."""
    down = torch.zeros(H, I).double()
    for h in range(H):
        at = torch.randperm(I, generator=gen)[:n]
        down[h, at] = torch.randint(0, 2, (n,), generator=gen).double() * 2 - 1
    return down


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [1, 9])
def test_past_the_range(T, eight):
    """Activations of up to a few million, weighed by both signs."""
    gen = torch.Generator().manual_seed(T)
    H, I = 80, 256
    case = Exact(whole(gen, 15, T, H - 1), torch.full((I,), 448.0).double(),
                 whole(gen, 15, I, H - 1), few(gen, H, I, 8), down_power=-9)
    assert (case.activations().abs() > 65520).double().mean() > 0.5
    case.check(eight)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [1, 9])
def test_low_in_the_range(T, eight):
    """Activations around 2^-16, whose low part alone would be below fp16's last bit."""
    gen = torch.Generator().manual_seed(T + 1)
    H, I = 80, 256
    case = Exact(whole(gen, 15, T, H - 1), torch.full((I,), 36.0).double(),
                 whole(gen, 15, I, H - 1), few(gen, H, I, 8), up_power=-22, x_power=-10,
                 down_power=6)
    a = case.activations().abs()
    assert float(a.max()) < 2.0 ** -12
    case.check(eight)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("power", [10, 15])
def test_large_beside_small(power, eight):
    """One activation far above its neighbours, which its outputs do not weigh."""
    gen = torch.Generator().manual_seed(power)
    H, I, T = 80, 256, 3
    up = whole(gen, 15, I, H - 1)
    up[:, 0] = 0
    up[::64] = 0
    up[::64, 0] = 8          # features 0, 64, ...: x's second input alone
    x = whole(gen, 15, T, H - 1)
    x[:, 0] = 2.0 ** power   # with the gate: 2^(power + 8) and more
    x[:, 1:] *= 2.0 ** -4
    down = few(gen, H, I, 8)
    down[:, ::64] = 0
    case = Exact(x, torch.full((I,), 32.0).double(), up, down, down_power=-5)
    a = case.activations().abs()
    assert (a[:, ::64] >= 2.0 ** (power + 8)).all()
    off = 2.0 ** -36 * float(a.max()) * 8 * 2.0 ** -5
    assert off < HALF      # of results around 1
    case.check(eight, off)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("I", [136, 144, 776])
def test_random_rows_past_the_range(I, eight):
    I = I // 16 * 16 if eight else I
    case = Layer("any", 6, 3, 5, 272, I, "fp16", eight)
    case.x = (case.x.float() * 1000).half()
    case.tw = case.tw * 2.0 ** -14
    case.args[1], case.args[2] = case.tw.cuda(), case.x.cuda()
    case.check(case.run())


@pytest.mark.parametrize("eight", [False, True])
def test_special_values_stay_in_their_token(eight):
    case = Layer("any", 6, 2, 4, 272, 48, "fp16", eight)
    clean = case.run()
    case.args[2][2, 7] = float("nan")
    case.args[2][4, 9] = float("inf")
    out = case.run()
    fine = torch.tensor([0, 1, 3, 5])
    assert torch.equal(out[fine], clean[fine])
    assert not out[2].isfinite().any() and not out[4].isfinite().any()
