"""The experts' products and activation against 64-bit references.

Every input's pad and tail rows hold NaN and every output is pre-filled with a
canary, so that an operand read from a row without a route, or a write outside
the documented rows, shows. Tolerances are bounds, not measurements:

- an output value passes one rounding to its type, at most half a step:
  eps/2 of the value (plus half the smallest subnormal);
- a sum of n terms held in fp32 is off by at most n steps of 2^-23 (twice the
  half step: a matrix instruction may truncate where an fp32 add rounds) of
  the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import combine_ep_prepare_amd as ep
import workloads
from combine_ep_prepare_amd import autograd as epa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CANARY = 1984.0   # exact in every payload type


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def route(kind, T, K, E, seed):
    """Routing tables by kind: distinct experts, some masked, all masked, all
    to one expert, the same expert twice, a steep load."""
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, K), E - 1, np.int64)
    if kind == "none":
        return np.full((T, K), -1, np.int64)
    if kind == "repeat":
        return np.repeat(rng.integers(0, E, (T, 1)), K, axis=1).astype(np.int64)
    if kind == "steep":
        idx = np.minimum(rng.geometric(0.5, (T, K)) - 1, E - 1)
        return idx.astype(np.int64)
    idx = np.argsort(rng.random((T, max(E, K))), axis=1)[:, :K].astype(np.int64)
    idx[idx >= E] = -1
    if kind == "masked":
        idx[rng.random((T, K)) < 0.6] = -1
    return idx


class Case:
    """One prepared routing and the live rows of each expert."""

    def __init__(self, kind, T, K, E, A, dtype, seed=0, cap=None, fill_pads=True,
                 zero_tail=False):
        self.dtype, self.E = DT[dtype], E
        self.eps2 = torch.finfo(self.dtype).eps / 2
        self.tiny = float(torch.finfo(self.dtype).smallest_normal) * self.eps2
        idx = route(kind, T, K, E, seed)
        self.cap = T * K + E * (A - 1) + 3 if cap is None else cap
        self.args = (T, K, E, A)
        self.flags = dict(fill_pads=fill_pads, zero_tail=zero_tail)
        L = self.layout(64)
        self.handle = ep.new_handle(L)
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        ep.prepare(L, torch.from_numpy(idx).cuda(), counts, self.handle, offsets)
        counts, offsets = counts.tolist(), offsets.tolist()
        assert counts == np.bincount(idx[idx >= 0], minlength=E).tolist()
        self.rows = [(o, max(o, min(o + n, self.cap))) for o, n in zip(offsets, counts)]
        self.total = min(offsets[E], self.cap)
        self.live = torch.zeros(self.cap, dtype=torch.bool)
        for a, b in self.rows:
            self.live[a:b] = True
        self.gen = torch.Generator().manual_seed(seed)

    def layout(self, H):
        T, K, E, A = self.args
        return ep.Layout(T, K, E, A, H, self.cap, dtype=self.dtype, **self.flags)

    def buffer(self, width, scale=1.0):
        """An expert-major input: values in live rows, NaN elsewhere."""
        t = (torch.randn(self.cap, width, generator=self.gen) * scale).to(self.dtype)
        t[~self.live] = float("nan")
        return t

    def weight(self, *shape):
        return (torch.randn(*shape, generator=self.gen) * shape[-1] ** -0.5).to(self.dtype)

    def out(self, *shape):
        return torch.full(shape, CANARY, dtype=self.dtype, device="cuda")

    def check_rows(self, got, want, bound, what):
        """got against the fp64 `want` within `bound` in live rows; zeros in
        pads and tail where the layout asks for them, else untouched."""
        got = got.cpu()
        filler = got[:self.total][~self.live[:self.total]]
        tail = got[self.total:]
        assert (filler == (0.0 if self.flags["fill_pads"] else CANARY)).all(), f"{what}: pads"
        assert (tail == (0.0 if self.flags["zero_tail"] else CANARY)).all(), f"{what}: tail"
        self.check(got[self.live], want[self.live], bound[self.live], what)

    def check(self, got, want, bound, what):
        got = got.double().cpu()
        assert torch.isfinite(got).all(), f"{what}: not finite"
        over = (got - want).abs() - (bound + self.eps2 * (want.abs() + bound) + self.tiny)
        assert got.numel() == 0 or over.max() <= 0, \
            f"{what}: {int((over > 0).sum())} values off, by up to {float(over.max())}"


def sum_bound(n, magnitudes):
    return n * 2.0 ** -23 * magnitudes


# kind, T, K, E, A, H, N: from nothing and one row to several tiles of every
# size the kernels use, with ragged rows, features and segments
SHAPES = [
    ("any", 0, 2, 3, 8, 64, 64),
    ("none", 40, 2, 3, 8, 64, 72),
    ("any", 1, 1, 1, 1, 8, 8),
    ("any", 1, 2, 5, 4, 264, 136),
    ("masked", 7, 3, 16, 1, 72, 1000),
    ("any", 33, 4, 6, 16, 520, 24),
    ("steep", 90, 2, 9, 1, 136, 264),
    ("repeat", 65, 4, 4, 2, 1032, 200),
    ("one", 257, 1, 3, 128, 192, 328),
    ("steep", 700, 2, 5, 16, 256, 520),
    ("any", 1100, 2, 4, 128, 328, 776),
    ("one", 515, 2, 2, 1, 72, 264),
    ("any", 640, 1, 2048, 1, 64, 64),
    # enough tiles for the larger ones: a few rows an expert, some, more than 128
    ("any", 700, 2, 64, 1, 648, 520),
    ("masked", 1300, 2, 64, 8, 520, 648),
    ("any", 8400, 2, 112, 1, 520, 520),
    ("steep", 9000, 2, 112, 4, 520, 776),
    # many rows an expert
    ("any", 3250, 4, 16, 8, 1032, 1048),
]
IDS = [f"{s[0]}-T{s[1]}E{s[3]}H{s[5]}N{s[6]}" for s in SHAPES]


def forward_reference(c, x, w):
    N = w.shape[1]
    want = torch.zeros(c.cap, N, dtype=torch.float64)
    mags = torch.zeros(c.cap, N, dtype=torch.float64)
    for e, (a, b) in enumerate(c.rows):
        xd, wd = x[a:b].double(), w[e].double()
        want[a:b] = xd @ wd.t()
        mags[a:b] = xd.abs() @ wd.abs().t()
    return want, mags


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_grouped_linear(shape, dtype):
    kind, T, K, E, A, H, N = shape
    c = Case(kind, T, K, E, A, dtype, zero_tail=H % 16 == 0)
    x, w, out = c.buffer(H), c.weight(E, N, H), c.out(c.cap, N)
    ep.grouped_linear(c.layout(H), c.handle, x.cuda(), w.cuda(), out)
    want, mags = forward_reference(c, x, w)
    c.check_rows(out, want, sum_bound(H, mags), "out")
    assert ep.read_status(c.handle) == 0


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_grouped_linear_bwd(shape, dtype):
    kind, T, K, E, A, H, N = shape
    c = Case(kind, T, K, E, A, dtype, fill_pads=H % 16 == 0)
    x, g, w = c.buffer(H), c.buffer(N), c.weight(E, N, H)
    gx, gw = c.out(c.cap, H), c.out(E, N, H)
    ep.grouped_linear_bwd(c.layout(H), c.handle, g.cuda(), x.cuda(), w.cuda(), gx, gw)
    want_x = torch.zeros(c.cap, H, dtype=torch.float64)
    mags_x = torch.zeros(c.cap, H, dtype=torch.float64)
    for e, (a, b) in enumerate(c.rows):
        gd, xd = g[a:b].double(), x[a:b].double()
        want_x[a:b] = gd @ w[e].double()
        mags_x[a:b] = gd.abs() @ w[e].double().abs()
        c.check(gw[e], gd.t() @ xd, sum_bound(b - a, gd.abs().t() @ xd.abs()),
                f"grad_weight[{e}]")
    c.check_rows(gx, want_x, sum_bound(N, mags_x), "grad_x")
    # each output alone gives the same bits, and leaves the other untouched
    gx1, gw1 = torch.empty_like(gx).fill_(CANARY), torch.empty_like(gw)
    ep.grouped_linear_bwd(c.layout(H), c.handle, g.cuda(), None, w.cuda(), gx1, None)
    ep.grouped_linear_bwd(c.layout(H), c.handle, g.cuda(), x.cuda(), None, None, gw1)
    assert torch.equal(gx1, gx) and torch.equal(gw1, gw)


def quantised(c, E, N, H, G, zeros):
    q = torch.randint(0, 256, (E, N, H // 2), generator=c.gen, dtype=torch.uint8)
    s = (torch.rand(E, N, H // G, generator=c.gen) * H ** -0.5 + 1e-3).to(c.dtype)
    z = torch.randint(0, 16, (E, N, H // G), generator=c.gen, dtype=torch.uint8) if zeros else None
    w = torch.stack((q & 15, q >> 4), dim=-1).reshape(E, N, H // G, G).double()
    zd = 8.0 if z is None else z.double()[..., None]
    w = (w - zd) * s.double()[..., None]
    return q, s, z, w.reshape(E, N, H)


QUANT = [
    ("any", 0, 2, 3, 8, 64, 64, 32), ("none", 9, 2, 3, 4, 64, 72, 64),
    ("any", 1, 1, 1, 1, 32, 8, 32), ("any", 1, 2, 8, 1, 1024, 520, 128),
    ("masked", 7, 3, 16, 1, 96, 1000, 32), ("any", 33, 4, 6, 16, 448, 24, 64),
    ("steep", 90, 2, 9, 1, 384, 264, 128), ("one", 17, 1, 3, 8, 2080, 136, 32),
    ("one", 300, 1, 2, 1, 640, 200, 128), ("repeat", 65, 4, 4, 2, 192, 88, 64),
    ("any", 40, 2, 300, 1, 256, 64, 128),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", QUANT, ids=[f"{s[0]}-T{s[1]}E{s[3]}H{s[5]}N{s[6]}G{s[7]}"
                                              for s in QUANT])
def test_grouped_linear_quant(shape, dtype, zeros):
    kind, T, K, E, A, H, N, G = shape
    c = Case(kind, T, K, E, A, dtype, zero_tail=True)
    x = c.buffer(H)
    q, s, z, w = quantised(c, E, N, H, G, zeros)
    out = c.out(c.cap, N)
    ep.grouped_linear_quant(c.layout(H), c.handle, x.cuda(), q.cuda(), s.cuda(),
                            None if z is None else z.cuda(), out)
    want, _ = forward_reference(c, x, w)
    # q enters the products with an offset that leaves the sum again by
    # (offset + z) * sum(x): 128 where the type holds 128..143 exactly (bf16),
    # 1024 where it holds 1024..1039 (fp16). A group's terms are bounded by
    # (offset + 15) + (offset + z) times |x| s, and pass G + 8 additions; the
    # groups' sums, at most 15 |x| s a term, pass H / G + 8 more.
    offset = 128.0 if dtype == "bf16" else 1024.0
    top = s.double().repeat_interleave(G, 2)
    bound = torch.zeros(c.cap, N, dtype=torch.float64)
    for e, (a, b) in enumerate(c.rows):
        mags = x[a:b].double().abs() @ top[e].t()
        bound[a:b] = sum_bound(G + 8, mags * (2 * offset + 30)) + sum_bound(H // G + 8, mags * 15)
    c.check_rows(out, want, bound, "out")
    # the bound above is for the worst order of roundings; over all values the
    # error stays within the type's own rounding plus a hundredth of a percent
    got = out.cpu()[c.live].double()
    off = (got - want[c.live]).norm()
    assert off <= (c.eps2 + 1e-4) * want[c.live].norm() + 1e-30


@pytest.mark.parametrize("fill,tail", [(True, False), (False, False), (True, True),
                                       (False, True)])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [("any", 0, 1, 2, 4, 8), ("none", 5, 2, 3, 4, 64),
                                   ("any", 1, 1, 1, 1, 8), ("masked", 61, 3, 7, 16, 264),
                                   ("steep", 400, 2, 6, 5, 1032)])
def test_swiglu(shape, dtype, fill, tail):
    kind, T, K, E, A, H = shape
    c = Case(kind, T, K, E, A, dtype, fill_pads=fill, zero_tail=tail)
    gu, grad = c.buffer(2 * H, 3.0), c.buffer(H)
    # far from zero on both sides, signed zeros and values next to zero
    odd = torch.tensor([0.0, -0.0, 1e-6, -1e-6, 30.0, -30.0, 200.0, -200.0]).to(c.dtype)
    live = c.live.nonzero().squeeze(1)
    if len(live):
        gu[live[0], :8] = odd
        gu[live[-1], H - 8:H] = odd
    L = c.layout(H)
    out, dgu = c.out(c.cap, H), c.out(c.cap, 2 * H)
    ep.swiglu(L, c.handle, gu.cuda(), out)
    ep.swiglu_bwd(L, c.handle, grad.cuda(), gu.cuda(), dgu)
    g, u, d = gu[:, :H].double(), gu[:, H:].double(), grad.double()
    s = torch.sigmoid(g)
    # a few fp32 operations on the way (exp, the quotient, four products and
    # two sums, each within two steps of its own value), 32 half steps in all;
    # s itself loses |g| half steps where exp's argument is rounded, and where
    # exp(-g) overflows fp32 (g < -88) s is 0 for a value below 2^-126
    rel = (32 + 2 * g.abs()) * 2.0 ** -24
    small = 2.0 ** -126 * (1 + g.abs()) * 2
    c.check_rows(out, g * s * u, rel * (g * s * u).abs() + small * u.abs(), "out")
    dg = s * (1 + g * (1 - s))
    want = torch.cat((d * u * dg, d * g * s), 1)
    # 1 + g (1 - s) cancels for negative g: its error is that of its terms
    terms = s * (1 + (g * (1 - s)).abs())
    bound = torch.cat(((rel * terms + small) * (d * u).abs(),
                       (rel * (g * s).abs() + small) * d.abs()), 1)
    c.check_rows(dgu, want, bound, "grad_gate_up")


@pytest.mark.parametrize("T", [5, 300, 1500])
def test_capacity_overflow(T):
    """Routes dropped past the capacity are no rows of any product."""
    H, N, E = 136, 264, 4
    worst = T * 2 + E * 7
    for cap in (0, 3, worst // 3, worst // 2):
        c = Case("any", T, 2, E, 8, "bf16", cap=cap)
        L = c.layout(H)
        x, g, w = c.buffer(H), c.buffer(N), c.weight(E, N, H)
        out, gx, gw = c.out(cap, N), c.out(cap, H), c.out(E, N, H)
        ep.grouped_linear(L, c.handle, x.cuda(), w.cuda(), out)
        ep.grouped_linear_bwd(L, c.handle, g.cuda(), x.cuda(), w.cuda(), gx, gw)
        want, mags = forward_reference(c, x, w)
        c.check_rows(out, want, sum_bound(H, mags), "out")
        assert torch.isfinite(gx.float()).all()
        for e, (a, b) in enumerate(c.rows):
            gd, xd = g[a:b].double(), x[a:b].double()
            c.check(gw[e], gd.t() @ xd, sum_bound(b - a, gd.abs().t() @ xd.abs()), "grad_weight")
        assert ep.read_status(c.handle) == ep.STATUS_OVERFLOW


@pytest.mark.parametrize("T", [6, 400])
def test_special_values_reach_exactly_their_outputs(T):
    """An infinity in one row reaches that row's outputs only; NaN weights of
    experts without rows reach none."""
    H, N, E = 128, 136, 4
    c = Case("one", T, 1, E, 1, "bf16", zero_tail=True)
    x, w = c.buffer(H), c.weight(E, N, H)
    a, b = c.rows[E - 1]
    x[a + 2, 5] = float("inf")
    x[a + 3, 7] = float("nan")
    w[:E - 1] = float("nan")
    w[E - 1, :, 5] = w[E - 1, :, 5].abs() + 0.5
    out, gw = c.out(c.cap, N), c.out(E, N, H)
    ep.grouped_linear(c.layout(H), c.handle, x.cuda(), w.cuda(), out)
    out = out.float().cpu()
    assert (out[a + 2] == float("inf")).all()
    assert out[a + 3].isnan().all()
    rest = [r for r in range(c.cap) if r not in (a + 2, a + 3)]
    assert torch.isfinite(out[rest]).all()
    bits = c.out(c.cap, N)
    ep.grouped_linear(c.layout(H), c.handle, x.cuda(), w.cuda(), bits)
    assert (bits[a + 3].view(torch.int16) == 0x7FC0).all()      # the canonical NaN
    g = c.buffer(N).cuda()
    ep.grouped_linear_bwd(c.layout(H), c.handle, g, x.cuda(), None, None, gw)
    gw = gw.float().cpu()
    assert (gw[:E - 1] == 0).all()
    bad = torch.zeros(H, dtype=torch.bool)
    bad[5] = bad[7] = True
    assert torch.isfinite(gw[E - 1][:, ~bad]).all()
    assert not torch.isfinite(gw[E - 1][:, bad]).any()


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 2.0 ** 127])
@pytest.mark.parametrize("zeros", [False, True])
def test_4_bit_special_values_stay_in_their_row(value, zeros):
    H, N, E, G, T = 256, 72, 4, 64, 37
    c = Case("one", T, 1, E, 8, "bf16", zero_tail=True)
    x = c.buffer(H)
    q, s, z, w = quantised(c, E, N, H, G, zeros)
    s[:E - 1] = float("nan")                     # experts without rows
    a = c.rows[E - 1][0]
    clean, dirty = c.out(c.cap, N), c.out(c.cap, N)
    args = [q.cuda(), s.cuda(), None if z is None else z.cuda()]
    ep.grouped_linear_quant(c.layout(H), c.handle, x.cuda(), *args, clean)
    x[a + 2, 5] = value
    ep.grouped_linear_quant(c.layout(H), c.handle, x.cuda(), *args, dirty)
    assert not torch.isfinite(dirty[a + 2].float()).any()
    keep = torch.arange(c.cap, device="cuda") != a + 2
    assert torch.isfinite(clean.float()).all() and torch.equal(clean[keep], dirty[keep])


def test_foreign_layout_writes_nothing():
    c = Case("any", 40, 2, 4, 8, "bf16")
    H = N = 64
    T, K, E, A = c.args
    L = ep.Layout(T, K, E, A * 2, H, c.cap)                     # not what was prepared
    x, w, s = c.buffer(H).cuda(), c.weight(E, N, H).cuda(), c.out(E, N, 2)
    q = torch.zeros(E, N, H // 2, dtype=torch.uint8, device="cuda")
    rows, wide, gw = c.out(c.cap, H), c.out(c.cap, 2 * H), c.out(E, N, H)
    calls = [lambda: ep.grouped_linear(L, c.handle, x, w, rows),
             lambda: ep.grouped_linear_bwd(L, c.handle, x, x, w, rows, gw),
             lambda: ep.grouped_linear_quant(L, c.handle, x, q, s, None, rows),
             lambda: ep.swiglu(L, c.handle, wide, rows),
             lambda: ep.swiglu_bwd(L, c.handle, x, wide, wide.clone())]
    for call in calls:
        call()
        assert ep.read_status(c.handle) == ep.STATUS_LAYOUT
        assert (rows == CANARY).all() and (gw == CANARY).all()


def test_rows_past_32_bit_offsets():
    """Rows and weights whose element offsets pass 2^31."""
    A, W, n = 300_000, 8192, 64
    idx = torch.tensor([[0], [1], [1], [1]], device="cuda")
    for H, N in ((n, W), (W, n)):
        L = ep.Layout(4, 1, 2, A, H, 2 * A, fill_pads=False)
        h = ep.new_handle(L)
        ep.prepare(L, idx, torch.empty(2, dtype=torch.int32, device="cuda"), h)
        x = torch.zeros(2 * A, H, dtype=torch.bfloat16, device="cuda")
        g = torch.zeros(2 * A, N, dtype=torch.bfloat16, device="cuda")
        x[A:A + 3].normal_()
        g[A:A + 3].normal_()
        w = (torch.randn(2, N, H, device="cuda") * H ** -0.5).bfloat16()
        out, gx, gw = torch.zeros_like(g), torch.zeros_like(x), torch.empty_like(w)
        ep.grouped_linear(L, h, x, w, out)
        ep.grouped_linear_bwd(L, h, g, x, w, gx, gw)
        xd, gd, wd = x[A:A + 3].double(), g[A:A + 3].double(), w[1].double()
        for got, want, mags, k in (
                (out[A:A + 3], xd @ wd.t(), xd.abs() @ wd.abs().t(), H),
                (gx[A:A + 3], gd @ wd, gd.abs() @ wd.abs(), N),
                (gw[1], gd.t() @ xd, gd.abs().t() @ xd.abs(), 3)):
            tol = sum_bound(k, mags) * 1.01 + 2.0 ** -8 * want.abs()
            assert ((got.double() - want).abs() <= tol).all()
        assert not out[:A].any() and not gx[A + 3:].any() and not gw[0].any()
        if H == n:
            q = torch.randint(0, 256, (2, N, H // 2), dtype=torch.uint8, device="cuda")
            s = torch.full((2, N, 1), 0.125, dtype=torch.bfloat16, device="cuda")
            out.zero_()
            ep.grouped_linear_quant(L, h, x, q, s, None, out)
            qd = torch.stack((q[1] & 15, q[1] >> 4), -1).reshape(N, H).double() - 8
            want = xd @ qd.t() * 0.125
            tol = sum_bound(H + 17, xd.abs().sum(1, keepdim=True) * 0.125 * 300)
            assert ((out[A:A + 3].double() - want).abs() <= tol * 1.01 + 2.0 ** -8 * want.abs()).all()
        else:
            gu = torch.zeros(2 * A, 2 * W, dtype=torch.bfloat16, device="cuda")
            gu[A:A + 3].normal_()
            act = torch.zeros_like(x)
            ep.swiglu(L, h, gu, act)
            a, b = gu[A:A + 3].double().chunk(2, 1)
            want = a * torch.sigmoid(a) * b
            assert ((act[A:A + 3].double() - want).abs() <= 2.0 ** -7.9 * want.abs() + 1e-30).all()
            del gu
        del x, g, w, out, gx, gw
        torch.cuda.empty_cache()


def test_weights_past_32_bit_offsets():
    E, N, H = 40, 8192, 8192
    idx = torch.tensor([[0, E - 1], [E - 1, 2]], device="cuda")
    L = ep.Layout(2, 2, E, 1, H, 4)
    h = ep.new_handle(L)
    ep.prepare(L, idx, torch.empty(E, dtype=torch.int32, device="cuda"), h)
    x = torch.randn(4, H, device="cuda").bfloat16()
    w = torch.empty(E, N, H, dtype=torch.bfloat16, device="cuda").normal_(0, H ** -0.5)
    out = torch.empty(4, N, dtype=torch.bfloat16, device="cuda")
    ep.grouped_linear(L, h, x, w, out)
    wd, xd = w[E - 1].double(), x[2:4].double()
    want, mags = xd @ wd.t(), xd.abs() @ wd.abs().t()
    tol = sum_bound(H, mags) * 1.01 + 2.0 ** -8 * want.abs()
    assert ((out[2:4].double() - want).abs() <= tol).all()
    gw = w
    ep.grouped_linear_bwd(L, h, out, x, None, None, gw)
    g = out[2:4].double()
    want, mags = g.t() @ xd, g.t().abs() @ xd.abs()
    assert ((gw[E - 1].double() - want).abs() <=
            sum_bound(2, mags) * 1.01 + 2.0 ** -8 * want.abs()).all()
    assert not gw[1].any() and not gw[E - 2].any()


# --------------------------------------------------------------------------
# together, as they are used
# --------------------------------------------------------------------------

def _mlp(x, w, idx, wgu, wd, E, A, H):
    routing = epa.EpRouting(idx, E, A, H)
    recv, recv_w = epa.dispatch(x, w, routing)
    hidden = epa.swiglu(epa.grouped_linear(recv, wgu, routing), routing)
    return epa.combine(epa.grouped_linear(hidden, wd, routing), routing, recv_w)


def _mlp64(x, w, idx, wgu, wd):
    out = torch.zeros_like(x)
    for e in range(wgu.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ wgu[e].t()).chunk(2, 1)
        out = out.index_add(0, t, w[t, k][:, None] * ((gate * torch.sigmoid(gate) * up)
                                                      @ wd[e].t()))
    return out


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K,E,A,H,I", [(1, 1, 2, 4, 64, 40), (50, 2, 6, 16, 128, 72),
                                         (900, 2, 5, 128, 264, 200)])
def test_expert_mlp_forward_and_gradients(T, K, E, A, H, I, dtype):
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(T)
    idx = torch.from_numpy(route("masked", T, K, E, T)).cuda()

    def leaf(*shape, scale=1.0):
        t = (torch.randn(*shape, generator=gen) * scale).to(dt)
        return t.cuda().requires_grad_(), t.double().requires_grad_()

    x, x64 = leaf(T, H)
    wgu, wgu64 = leaf(E, 2 * I, H, scale=H ** -0.5)
    wd, wd64 = leaf(E, H, I, scale=I ** -0.5)
    w = torch.rand(T, K, generator=gen)
    w64 = w.double().requires_grad_()
    w = w.cuda().requires_grad_()
    grad = torch.randn(T, H, generator=gen).to(dt)
    y = _mlp(x, w, idx, wgu, wd, E, A, H)
    y.backward(grad.cuda())
    y64 = _mlp64(x64, w64, idx.cpu(), wgu64, wd64)
    y64.backward(grad.double())
    # at most seven roundings to the type lie on a value's way through the
    # chain and back, each half a step of its own tensor's values; in the
    # 2-norm they add up to at most that many half steps, times four for the
    # products that carry them on (the activation's slopes are below 1.1, the
    # weights are scaled to keep norms, and up to K * 2 paths meet)
    tol = 4 * 7 * torch.finfo(dt).eps / 2 + 2000 * 2.0 ** -23
    for name, got, want in (("y", y, y64), ("x", x.grad, x64.grad), ("w", w.grad, w64.grad),
                            ("wgu", wgu.grad, wgu64.grad), ("wd", wd.grad, wd64.grad)):
        off = (got.detach().double().cpu() - want.detach()).norm()
        assert off <= tol * want.norm() + 1e-30, (name, float(off), float(want.norm()))


def test_gradients_against_differences():
    """fp32, a central difference of the whole chain along random directions."""
    T, K, E, A, H, I = 37, 2, 4, 8, 64, 48
    gen = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.from_numpy(route("any", T, K, E, 3)).cuda()

    def leaf(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).requires_grad_()

    leaves = [leaf(T, H), leaf(T, K), leaf(E, 2 * I, H, scale=H ** -0.5),
              leaf(E, H, I, scale=I ** -0.5)]
    probe = torch.randn(T, H, generator=gen, device="cuda").double()

    def value(ls):
        x, w, a, b = ls
        return (_mlp(x, w, idx, a, b, E, A, H).double() * probe).sum()

    _mlp(*leaves[:2], idx, *leaves[2:], E, A, H).backward(probe.float())
    with torch.no_grad():
        for i, p in enumerate(leaves):
            v = torch.randn(p.shape, generator=gen, device="cuda")
            v /= v.norm()
            h = 2.0 ** -5
            plus, minus = ([q + s * h * v if j == i else q for j, q in enumerate(leaves)]
                           for s in (1, -1))
            diff = (value(plus) - value(minus)) / (2 * h)
            slope = (p.grad.double() * v.double()).sum()
            # rounding: 2^-24 of a value of norm ~|probe||y|, over 2h; curvature: h^2/6 of a
            # third derivative along a unit direction, below the first's own scale
            scale = p.grad.double().norm()
            assert abs(diff - slope) <= 2e-3 * scale + 1e-3, (i, float(diff), float(slope))


def test_decode_chain_with_4_bit_weights():
    T, K, E, H, I, G = 6, 2, 12, 256, 128, 64
    c = Case("any", T, K, E, 1, "bf16")
    idx = torch.from_numpy(route("any", T, K, E, 0)).cuda()
    q1, s1, z1, w1 = quantised(c, E, 2 * I, H, G, True)
    q2, s2, z2, w2 = quantised(c, E, H, I, G, False)
    x = torch.randn(T, H, generator=c.gen).bfloat16()
    w = torch.rand(T, K, generator=c.gen)
    routing = epa.EpRouting(idx, E, 1, H)
    with torch.no_grad():
        recv, recv_w = epa.dispatch(x.cuda(), w.cuda(), routing)
        hid = epa.grouped_linear_quant(recv, q1.cuda(), s1.cuda(), routing, z1.cuda())
        y = epa.grouped_linear_quant(epa.swiglu(hid, routing), q2.cuda(), s2.cuda(), routing)
        out = epa.combine(y, routing, recv_w)
    want = _mlp64(x.double(), w.double(), idx.cpu(), w1, w2)
    # four roundings to bf16 on the way, as above
    assert (out.double().cpu() - want).norm() <= 4 * 4 * 2.0 ** -8 * want.norm()


def test_same_bits_every_time_and_on_another_stream():
    c = Case("steep", 700, 2, 5, 16, "bf16", zero_tail=True)
    H, N = 264, 520
    L = c.layout(H)
    x, g, w = c.buffer(H).cuda(), c.buffer(N).cuda(), c.weight(5, N, H).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = None
    for stream in (None, side, None, side):
        out, gx, gw = c.out(c.cap, N), c.out(c.cap, H), c.out(5, N, H)
        torch.cuda.synchronize()
        ep.grouped_linear(L, c.handle, x, w, out, stream=stream)
        ep.grouped_linear_bwd(L, c.handle, g, x, w, gx, gw, stream=stream)
        torch.cuda.synchronize()
        if first is None:
            first = (out, gx, gw)
        assert all(torch.equal(a, b) for a, b in zip(first, (out, gx, gw)))


def test_captured_and_replayed():
    """Prepare and every expert op in one graph, replayed on new routings and
    values with eager work between the replays."""
    T, K, E, A, H, I, G = 96, 2, 6, 8, 128, 64, 32
    cap = T * K + E * (A - 1)
    L, LI = (ep.Layout(T, K, E, A, n, cap, zero_tail=True) for n in (H, I))
    idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
    x = torch.empty(cap, H, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn(E, 2 * I, H, device="cuda", generator=gen) * H ** -0.5).bfloat16()
    q = torch.randint(0, 256, (E, 2 * I, H // 2), device="cuda", generator=gen, dtype=torch.uint8)
    s = torch.full((E, 2 * I, H // G), 0.02, dtype=torch.bfloat16, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")

    def outputs():
        return [torch.empty(n, m, dtype=torch.bfloat16, device="cuda") for n, m in
                ((cap, 2 * I), (cap, I), (cap, 2 * I), (cap, H), (E * 2 * I, H), (cap, 2 * I))]

    def step(handle, o):
        ep.prepare(L, idx, counts, handle)
        ep.grouped_linear(L, handle, x, w, o[0])
        ep.swiglu(LI, handle, o[0], o[1])
        ep.swiglu_bwd(LI, handle, o[1], o[0], o[2])
        ep.grouped_linear_bwd(L, handle, o[2], x, w, o[3], o[4].view(E, 2 * I, H))
        ep.grouped_linear_quant(L, handle, x, q, s, None, o[5])

    def fill(i):
        idx.copy_(torch.from_numpy(route(("any", "masked", "one", "none", "steep")[i % 5], T, K,
                                         E, i)))
        x.normal_(generator=gen)

    fill(0)
    handle, o = ep.new_handle(L), outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(handle, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(handle, o)
    h2, o2 = ep.new_handle(L), outputs()
    for i in range(1, 8):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        step(h2, o2)
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(o, o2)):
            assert torch.equal(a, b), (i, k)


def test_captured_training_step():
    """A whole autograd step in one graph: the leaves' gradients after each
    replay against an eager step on the same values."""
    T, K, E, A, H, I = 96, 2, 6, 8, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(T, K, device="cuda")
    idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
    weights = [(torch.randn(E, a, b, device="cuda", generator=gen) * b ** -0.5).bfloat16()
               for a, b in ((2 * I, H), (H, I))]

    def fill(i):
        idx.copy_(torch.from_numpy(route(("any", "masked", "steep")[i % 3], T, K, E, i)))
        x.normal_(generator=gen)
        w.uniform_(generator=gen)

    def leaves():
        return [x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_(),
                *(p.clone().requires_grad_() for p in weights)]

    def grads(ls):
        y = _mlp(ls[0], ls[1], idx, ls[2], ls[3], E, A, H)
        return torch.autograd.grad(y.float().square().sum(), ls)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(leaves())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = grads(leaves())
    for i in range(1, 7):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(captured, grads(leaves()))):
            assert torch.equal(a, b), (i, k)


def test_two_streams_at_once():
    """Two routings' products in flight on two streams, in each kernel that a
    product may take."""
    H, N = 264, 520
    cases = [Case(kind, T, 2, E, 4, "bf16", seed=T, zero_tail=True)
             for kind, T, E in (("any", 40, 8), ("steep", 900, 8), ("any", 8400, 112))]
    for c in cases:
        c.x, c.w = c.buffer(H).cuda(), c.weight(c.E, N, H).cuda()
        c.alone = c.out(c.cap, N)
        ep.grouped_linear(c.layout(H), c.handle, c.x, c.w, c.alone)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[c.out(c.cap, N) for _ in range(3)] for c in cases]
    torch.cuda.synchronize()
    for i in range(3):
        for c, st, o in zip(cases, streams, outs):
            ep.grouped_linear(c.layout(H), c.handle, c.x, c.w, o[i], stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        assert all(torch.equal(t, c.alone) for t in o)


def test_custom_ops_match_the_binding():
    import combine_ep_prepare_amd.custom_ops as co
    T, K, E, A, H, I = 60, 2, 5, 8, 64, 32
    cap = T * K + E * (A - 1)
    L = ep.Layout(T, K, E, A, H, cap)
    ll, handle = co.layout_list(L), ep.new_handle(L)
    co.prepare(torch.from_numpy(route("any", T, K, E, 0)).cuda(), handle, ll)
    x = torch.randn(cap, H, device="cuda").bfloat16().requires_grad_()
    w = (torch.randn(E, 2 * I, H, device="cuda") / 8).bfloat16().requires_grad_()
    y = co.swiglu(co.grouped_linear(x, w, handle, ll), handle, ll)
    grad = torch.randn_like(y)
    y.backward(grad)
    LI, LT = ep.Layout(T, K, E, A, I, cap, zero_tail=True), ep.Layout(T, K, E, A, H, cap,
                                                                      zero_tail=True)
    a, b, c = (torch.empty(cap, n, dtype=torch.bfloat16, device="cuda") for n in (2 * I, I, 2 * I))
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    with torch.no_grad():
        ep.grouped_linear(LT, handle, x, w, a)
        ep.swiglu(LI, handle, a, b)
        ep.swiglu_bwd(LI, handle, grad, a, c)
        ep.grouped_linear_bwd(LT, handle, c, x, w, gx, gw)
    assert torch.equal(y, b) and torch.equal(x.grad, gx) and torch.equal(w.grad, gw)
    q = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device="cuda")
    s = torch.rand(E, 2 * I, H // 32, device="cuda").bfloat16()
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda")
    torch.library.opcheck(co.grouped_linear_quant, (x.detach(), q, s, z, handle, ll))
    torch.library.opcheck(co.swiglu, (a.detach().requires_grad_(), handle, ll))
    torch.library.opcheck(co.grouped_linear, (x, w, handle, ll))


def test_expanded_and_strided_inputs():
    """The autograd ops take gradients and inputs that are not contiguous."""
    T, K, E, H, I = 40, 2, 4, 64, 32
    idx = torch.from_numpy(route("any", T, K, E, 0)).cuda()
    routing = epa.EpRouting(idx, E, 4, H)
    cap = routing.layout.cap
    wide = torch.randn(cap, 2 * H, device="cuda").bfloat16()
    w = (torch.randn(E, H, 2 * I, device="cuda") / 8).bfloat16()
    x = wide[:, ::2].requires_grad_()
    wt = w.transpose(1, 2).requires_grad_()
    y = epa.swiglu(epa.grouped_linear(x, wt, routing), routing)
    y.backward(torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand_as(y))
    x2, w2 = x.detach().contiguous().requires_grad_(), wt.detach().contiguous().requires_grad_()
    y2 = epa.swiglu(epa.grouped_linear(x2, w2, routing), routing)
    y2.backward(torch.ones_like(y2))
    assert torch.equal(y, y2) and torch.equal(x.grad, x2.grad) and torch.equal(wt.grad, w2.grad)


def test_second_derivatives_are_refused():
    T, K, E, H, I = 40, 2, 4, 64, 32
    routing = epa.EpRouting(torch.from_numpy(route("any", T, K, E, 0)).cuda(), E, 4, H)
    x = torch.randn(routing.layout.cap, H, device="cuda").requires_grad_()
    w = torch.randn(E, 2 * I, H, device="cuda").requires_grad_()
    y = epa.grouped_linear(x, w, routing)
    for of, name in ((y, "grouped_linear"), (epa.swiglu(y, routing), "swiglu")):
        with pytest.raises(RuntimeError, match=f"{name} has no second derivative"):
            torch.autograd.grad(of.square().sum(), x, create_graph=True)


def test_share_of_a_workload():
    """A slice of the masked workload through both products, against fp64 on
    the GPU."""
    cfg = workloads.scaled(workloads.CONFIGS["masked"], T=2048, H=512)
    r = workloads.make_routing(cfg)
    routing = epa.EpRouting(torch.from_numpy(r.topk_idx).cuda(), cfg.E, cfg.A, cfg.H)
    x = workloads.randn_bf16_torch((cfg.T, cfg.H), 3)
    w = torch.from_numpy(r.topk_weights).cuda()
    wt = (torch.randn(cfg.E, 264, cfg.H, device="cuda") * cfg.H ** -0.5).bfloat16()
    recv, _ = epa.dispatch(x, w, routing)
    out = epa.grouped_linear(recv, wt, routing)
    off, n = routing.expert_offsets.tolist(), routing.token_counts.tolist()
    for e in range(cfg.E):
        a, b = off[e], off[e] + n[e]
        xd, wd = recv[a:b].double(), wt[e].double()
        want, mags = xd @ wd.t(), xd.abs() @ wd.abs().t()
        tol = sum_bound(cfg.H, mags) * 1.01 + 2.0 ** -8 * want.abs()
        assert ((out[a:b].double() - want).abs() <= tol).all()
        assert not out[b:off[e + 1]].any()
