"""The experts' ops at the ends of what their documentation allows."""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_experts import Case, quantised, sum_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def prepared(idx, E, H, cap, A=1, **kw):
    T, K = idx.shape
    L = ep.Layout(T, K, E, A, H, cap, **kw)
    handle = ep.new_handle(L)
    ep.prepare(L, idx.cuda(), torch.empty(E, dtype=torch.int32, device="cuda"), handle)
    return L, handle


def test_weight_gradient_of_more_tiles_than_a_grid_direction_holds():
    """2048 experts of 8 x 2^20 weights: 2^24 tiles of 256 threads each, one more
    than 2^32 - 1 threads hold."""
    E, N, H = 2048, 8, 1 << 20
    first, last = 5, E - 1
    L, handle = prepared(torch.tensor([[last], [first], [last]]), E, H, 3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, H, device="cuda", generator=gen).bfloat16()
    g = torch.randn(3, N, device="cuda", generator=gen).bfloat16()
    gw = torch.full((E, N, H), 3.0, dtype=torch.bfloat16, device="cuda")
    ep.grouped_linear_bwd(L, handle, g, x, None, None, gw)
    for e, a, b in ((first, 0, 1), (last, 1, 3)):
        gd, xd = g[a:b].double(), x[a:b].double()
        want, mags = gd.t() @ xd, gd.t().abs() @ xd.abs()
        # two fp32 roundings of the sum, one to bf16
        tol = 2 * 2.0 ** -23 * mags * 1.01 + 2.0 ** -8 * want.abs()
        assert ((gw[e].double() - want).abs() <= tol).all()
    for part in (gw[:first], gw[first + 1:1024], gw[1024:last]):
        assert not part.any()


# --------------------------------------------------------------------------
# refusals, each call by itself
# --------------------------------------------------------------------------

FOREIGN = ["grouped_linear", "grad_x", "grad_weight", "few rows", "quant", "swiglu", "swiglu_bwd"]


@pytest.mark.parametrize("call", FOREIGN)
def test_foreign_layout_is_refused_by_each_call(call):
    """A handle prepared for another layout: the status bit, set by this very
    call, and no output touched."""
    T, K, E, A, H, N = 300, 2, 4, 8, 64, 72
    cap = T * K + E * (A - 1)
    idx = torch.arange(T * K).reshape(T, K) % E
    _, handle = prepared(idx, E, H, cap, A)
    assert ep.read_status(handle) == 0
    T = 20 if call == "few rows" else T                      # not the tokens of the handle
    L = ep.Layout(T, K, E, A * 2, H, cap, zero_tail=True)
    x, g, gu = (torch.ones(cap, n, dtype=torch.bfloat16, device="cuda") for n in (H, N, 2 * H))
    w = torch.ones(E, N, H, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(E, N, H // 2, dtype=torch.uint8, device="cuda")
    s = torch.ones(E, N, H // 32, dtype=torch.bfloat16, device="cuda")
    shape = {"grad_x": (cap, H), "grad_weight": (E, N, H), "swiglu": (cap, H),
             "swiglu_bwd": (cap, 2 * H)}.get(call, (cap, N))
    out = torch.full(shape, 1984.0, dtype=torch.bfloat16, device="cuda")
    {"grouped_linear": lambda: ep.grouped_linear(L, handle, x, w, out),
     "few rows": lambda: ep.grouped_linear(L, handle, x, w, out),
     "grad_x": lambda: ep.grouped_linear_bwd(L, handle, g, None, w, out, None),
     "grad_weight": lambda: ep.grouped_linear_bwd(L, handle, g, x, None, None, out),
     "quant": lambda: ep.grouped_linear_quant(L, handle, x, q, s, None, out),
     "swiglu": lambda: ep.swiglu(L, handle, gu, out),
     "swiglu_bwd": lambda: ep.swiglu_bwd(L, handle, x, gu, out)}[call]()
    assert ep.read_status(handle) == ep.STATUS_LAYOUT
    assert (out == 1984.0).all()


# --------------------------------------------------------------------------
# routes dropped past the capacity
# --------------------------------------------------------------------------

@pytest.mark.parametrize("fill,tail", [(True, False), (False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [5, 300, 1500])
def test_every_op_past_the_capacity(T, dtype, fill, tail):
    H, N, E, G = 128, 264, 4, 32
    worst = T * 2 + E * 7
    for cap in (0, 3, worst // 3, worst // 2):
        c = Case("any", T, 2, E, 8, dtype, cap=cap, fill_pads=fill, zero_tail=tail)
        L = c.layout(H)
        g, w, gu, d = c.buffer(N), c.weight(E, N, H), c.buffer(2 * H), c.buffer(H)
        gx, act, dgu = c.out(cap, H), c.out(cap, H), c.out(cap, 2 * H)
        ep.grouped_linear_bwd(L, c.handle, g.cuda(), None, w.cuda(), gx, None)
        want, mags = (torch.zeros(cap, H, dtype=torch.float64) for _ in range(2))
        for e, (a, b) in enumerate(c.rows):
            want[a:b] = g[a:b].double() @ w[e].double()
            mags[a:b] = g[a:b].double().abs() @ w[e].double().abs()
        c.check_rows(gx, want, sum_bound(N, mags), "grad_x")
        ep.swiglu(L, c.handle, gu.cuda(), act)
        ep.swiglu_bwd(L, c.handle, d.cuda(), gu.cuda(), dgu)
        a, b, dd = gu[:, :H].double(), gu[:, H:].double(), d.double()
        s, rest = torch.sigmoid(a), torch.sigmoid(-a)
        # 42 units of 2^-24 and the exponent's |g|, below 8 here, of the terms
        unit = 52 * 2.0 ** -24
        c.check_rows(act, a * s * b, unit * (a * s * b).abs(), "swiglu")
        want = torch.cat((dd * b * s * (1 + a * rest), dd * a * s), 1)
        mags = torch.cat(((dd * b * s).abs() * (1 + (a * rest).abs()), (dd * a * s).abs()), 1)
        c.check_rows(dgu, want, unit * mags, "swiglu_bwd")
        if dtype != "fp32":
            out = c.out(cap, N)
            x = c.buffer(H)
            q, sc, z, wq = quantised(c, E, N, H, G, True)
            ep.grouped_linear_quant(L, c.handle, x.cuda(), q.cuda(), sc.cuda(), z.cuda(), out)
            want, mags = torch.zeros(cap, N, dtype=torch.float64), torch.zeros(cap, N,
                                                                              dtype=torch.float64)
            for e, (lo, hi) in enumerate(c.rows):
                xd = x[lo:hi].double()
                want[lo:hi] = xd @ wq[e].t()
                # operands up to 31 and a start of up to 31 times the sum of x
                mags[lo:hi] = xd.abs() @ sc[e].double().repeat_interleave(G, 1).t() * 62
            c.check_rows(out, want, sum_bound(G + H // G + 16, mags), "quant")
        assert ep.read_status(c.handle) == ep.STATUS_OVERFLOW


# --------------------------------------------------------------------------
# weights past 2^31 elements, values at the ends of a type
# --------------------------------------------------------------------------

def test_tiles_of_weights_past_32_bit_offsets():
    """40 experts of 8192 x 8192: the last one's weights lie past 2^31 elements;
    twenty rows an expert on average, so that both products take tiles."""
    E, N, H, T = 40, 8192, 8192, 800
    idx = torch.where(torch.arange(T) % 20 == 0, E - 1, 3)[:, None]
    L, handle = prepared(idx, E, H, T)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, g = (torch.randn(T, n, device="cuda", generator=gen).bfloat16() for n in (H, N))
    w = torch.empty(E, N, H, dtype=torch.bfloat16, device="cuda")
    w[3].normal_(0, H ** -0.5, generator=gen)
    w[E - 1].normal_(0, H ** -0.5, generator=gen)
    out, gx = torch.empty_like(g), torch.empty_like(x)
    ep.grouped_linear(L, handle, x, w, out)
    ep.grouped_linear_bwd(L, handle, g, None, w, gx, None)
    n = T // 20
    for e, a, b in ((3, 0, T - n), (E - 1, T - n, T)):
        wd = w[e].double()
        for got, lhs, rhs in ((out[a:b], x[a:b].double(), wd.t().contiguous()),
                              (gx[a:b], g[a:b].double(), wd)):
            want, mags = lhs @ rhs, lhs.abs() @ rhs.abs()
            tol = sum_bound(H, mags) * 1.01 + 2.0 ** -8 * want.abs()
            assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [6, 200])
def test_subnormal_operands_count(T, dtype):
    """Operands below the smallest normal number, times large ones."""
    H, N, E = 64, 72, 2
    c = Case("one", T, 1, E, 1, dtype)
    info = torch.finfo(c.dtype)
    step = float(info.smallest_normal) * info.eps
    gen = c.gen
    small = (torch.randint(1, 4, (c.cap, H), generator=gen) * step).to(c.dtype)
    assert (small.double() > 0).all() and (small.double() < info.smallest_normal).all()
    large = (torch.randint(1, 9, (E, N, H), generator=gen) * 2.0 ** (
        10 if dtype == "fp16" else 100)).to(c.dtype)
    out, gx, gw = c.out(c.cap, N), c.out(c.cap, H), c.out(E, N, H)
    x = small.clone()
    x[~c.live] = float("nan")
    g = c.buffer(N)
    L = c.layout(H)
    ep.grouped_linear(L, c.handle, x.cuda(), large.cuda(), out)
    ep.grouped_linear_bwd(L, c.handle, (g * 64).to(c.dtype).cuda(), x.cuda(), None, None, gw)
    ep.grouped_linear_bwd(L, c.handle, g.cuda(), None, (large * 0 + small[:1, :H]).cuda(), gx, None)
    a, b = c.rows[E - 1]
    xd, wd, gd = x[a:b].double(), large[E - 1].double(), (g * 64).to(c.dtype)[a:b].double()
    # sums of whole multiples of the steps: exact up to the one rounding, but for
    # the gradients' general factor, and to fp32's own smallest step
    for got, want, mags, n in ((out[a:b], xd @ wd.t(), None, 0),
                               (gw[E - 1], gd.t() @ xd, gd.abs().t() @ xd, b - a),
                               (gx[a:b], g[a:b].double() @ small[:1].double().expand(N, H),
                                g[a:b].double().abs() @ small[:1].double().expand(N, H), N)):
        bound = 0 if mags is None else sum_bound(n, mags) + n * 2.0 ** -149
        tol = bound + c.eps2 * want.abs() * 1.01 + step
        assert ((got.double().cpu() - want).abs() <= tol).all()
    assert (out[a:b] != 0).all() and (gw[E - 1] != 0).float().mean() > 0.5
