"""The layer for a few tokens against 64-bit references.

Bounds, step by step: the first product's sums (n steps of 2^-23 of the terms'
magnitudes for n terms, and 4 steps more a block of scaled weights); the activation,
whose slope in the gate is below 1.1 of |up| and in up |silu|, 24 + 2 |gate| units of
2^-24 of its own (the exponent's rounding grows with the gate), held as the sum of
two values of the payload type: half a step of half a step off; the second product's
sums, of twice as many terms, off by that; K weighted terms in fp32; one rounding.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from combine_ep_prepare_amd import autograd as epa
from test_gpu_experts import DT, route
from test_gpu_norm import U
from test_gpu_scaled import weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    def __init__(self, kind, T, K, E, H, I, dtype, eight, seed=0):
        self.dt, self.eight, self.K, self.E, self.H, self.I = DT[dtype], eight, K, E, H, I
        gen = torch.Generator().manual_seed(seed + T + H)
        self.idx = torch.from_numpy(route(kind, T, K, E, seed + T)).contiguous()
        self.tw = torch.randn(T, K, generator=gen)
        self.x = torch.randn(T, H, generator=gen).to(self.dt)
        if eight:
            (self.gu, self.gus, self.guv) = weights(gen, E, 2 * I, H)
            (self.dn, self.dns, self.dnv) = weights(gen, E, H, I)
        else:
            self.gu = (torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5).to(self.dt)
            self.dn = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(self.dt)
            self.gus = self.dns = None
            self.guv, self.dnv = self.gu.double(), self.dn.double()
        self.layout = ep.Layout(T, K, E, 1, H, 0, dtype=self.dt)
        self.args = [t if t is None else t.cuda() for t in
                     (self.idx, self.tw, self.x, self.gu, self.dn, self.gus, self.dns)]
        self.workspace = ep.new_expert_layer_workspace(self.layout, I).fill_(255)

    def run(self, out=None):
        out = torch.full_like(self.x, 7.0, device="cuda") if out is None else out
        idx, tw, x, gu, dn, gus, dns = self.args
        ep.expert_layer(self.layout, idx, tw, x, gu, dn, out, self.workspace, gus, dns)
        return out

    def want(self):
        H, I, half = self.H, self.I, torch.finfo(self.dt).eps / 2
        tiny = torch.finfo(self.dt).smallest_normal * half
        T = self.x.shape[0]
        want, bound = (torch.zeros(T, H, dtype=torch.float64) for _ in range(2))
        n1, n2 = H + 4 * (-(-H // 128)), 2 * I + 4 * (-(-I // 128))
        for e in range(self.E):
            t, k = (self.idx == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            x, w1, w2 = self.x[t].double(), self.guv[e], self.dnv[e]
            g, u = (x @ w1.t()).chunk(2, 1)
            eg, eu = (n1 * 2.0 ** -23 * (x.abs() @ w1.abs().t())).chunk(2, 1)
            a = g * torch.sigmoid(g) * u
            silu = (g * torch.sigmoid(g)).abs()
            ea = 1.1 * eg * (u.abs() + eu) + silu * eu + (24 + 2 * g.abs()) * U * a.abs()
            ea = ea + half * half * (a.abs() + ea) + tiny
            y, mag = a @ w2.t(), (a.abs() + ea) @ w2.abs().t()
            ey = ea @ w2.abs().t() + n2 * 2.0 ** -23 * mag
            w = self.tw[t, k].double()[:, None]
            want.index_add_(0, t, w * y)
            bound.index_add_(0, t, w.abs() * (ey + self.K * 2 * U * mag))
        return want, bound + half * (want.abs() + bound) + tiny

    def check(self, out):
        want, bound = self.want()
        off = (out.double().cpu() - want).abs()
        assert out.isfinite().all() and (off <= bound).all(), float((off - bound).max())


CASES = [("any", 1, 1, 1, 16, 16), ("any", 1, 2, 8, 256, 128), ("any", 3, 2, 5, 1040, 272),
         ("masked", 16, 8, 64, 512, 144), ("none", 4, 2, 3, 64, 64), ("one", 40, 1, 3, 144, 208),
         ("repeat", 9, 4, 6, 272, 400), ("steep", 64, 8, 128, 256, 64), ("any", 33, 1, 40, 128, 1040),
         ("any", 1, 8, 256, 2048, 768), ("any", 512, 2, 2048, 64, 32), ("one", 16, 64, 2, 80, 96),
         ("any", 64, 16, 16, 208, 144)]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind,T,K,E,H,I", CASES)
def test_layer(kind, T, K, E, H, I, dtype, eight):
    case = Layer(kind, T, K, E, H, I, dtype, eight)
    out = case.run()
    case.check(out)
    # the same bits again, from a workspace that holds the last call's values
    assert torch.equal(case.run(), out)


@pytest.mark.parametrize("H,I", [(8, 8), (72, 24), (1032, 776), (264, 40)])
def test_odd_sizes(H, I):
    case = Layer("masked", 5, 3, 7, H, I, "fp16", False)
    case.check(case.run())


def test_ids_outside_count_nothing():
    case = Layer("any", 6, 3, 5, 64, 48, "bf16", False)
    out = case.run()
    bad = case.args[0].clone()
    keep = torch.ones(6, 3, dtype=torch.bool)
    for at, v in (((0, 1), 5), ((1, 0), -7), ((2, 2), 1 << 40), ((3, 1), -(1 << 62)), ((4, 0), 2048)):
        bad[at] = v
        keep[at] = False
    bad[5] = 100
    keep[5] = False
    case.args[0] = bad
    got = case.run()
    case.idx = torch.where(keep, case.idx, -1)
    case.check(got)
    assert (got[5] == 0).all() and not torch.equal(got, out)


def test_special_values_stay_in_their_token():
    case = Layer("any", 6, 2, 4, 272, 48, "bf16", True)
    case.args[2][2, 7] = float("nan")
    case.args[2][4, 9] = float("inf")
    out = case.run()
    fine = torch.tensor([0, 1, 3, 5])
    assert out[fine].isfinite().all() and not out[2].isfinite().any() and not out[4].isfinite().any()


def test_two_streams():
    """Two calls at once, each with a workspace of its own."""
    a, b = (Layer("any", 8, 4, 16, 512, 256, "bf16", True, seed=s) for s in (1, 2))
    want = a.run(), b.run()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for case, out, s in zip((a, b), outs, streams):
            with torch.cuda.stream(s):
                case.run(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_captured():
    case = Layer("masked", 4, 3, 6, 144, 80, "bf16", False)
    want = case.run()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.run(out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        # other routes in the same place
    case.args[0].copy_(torch.from_numpy(route("any", 4, 3, 6, 99)).cuda())
    case.idx = case.args[0].cpu()
    graph.replay()
    case.check(out)


@pytest.mark.parametrize("eight", [False, True])
def test_like_the_routed_path(eight):
    """The same layer by prepare, dispatch, the products and combine (16 bits), and
    through the differentiable module."""
    case = Layer("any", 12, 3, 9, 256, 128, "bf16", eight)
    idx, tw, x, gu, dn, gus, dns = case.args
    out = epa.expert_layer(x, idx, tw, gu, dn, gus, dns)
    assert torch.equal(out, case.run())
    if eight:
        return
    routing = epa.EpRouting(idx, 9, 1, 256)
    recv, rw = epa.dispatch(x, tw, routing)
    act = epa.swiglu(epa.grouped_linear(recv, gu, routing), routing)
    y = epa.combine(epa.grouped_linear(act, dn, routing), routing, rw)
    # the routed path rounds gate, up and each product too
    assert (out.double() - y.double()).norm() <= 0.02 * y.double().norm()
    with pytest.raises(RuntimeError, match="no backward"):
        epa.expert_layer(x.clone().requires_grad_(), idx, tw, gu, dn)
