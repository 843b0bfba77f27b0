"""The norm in front of a layer against 64-bit references.

Tolerances are bounds, not measurements. u = 2^-24 is half a step of fp32 relative
to the value:
- the sum of squares: a lane chains up to 32 fused multiply-adds, then up to 6
  exchanges and 16 partial sums: within 64 u of its value (all terms are positive);
- r, its inverse root: half of that, and a handful of roundings: 40 u;
- a result is two more products: 48 u of its value, then one rounding to its
  type, at most half a step;
- in 8 bits: q is off y / scale by half a step of e4m3: 2^-4 of the value, or 2^-10
  below 2^-6, where steps are 2^-9.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from combine_ep_prepare_amd import autograd as epa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
EPS = 1e-6
LEAST = 448.0 * 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rounded(want, bound, dtype):
    """What a value within `bound` of want may be after its one rounding."""
    half = torch.finfo(dtype).eps / 2
    return bound + half * (want.abs() + bound) + torch.finfo(dtype).smallest_normal * half


def values(T, H, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=gen) * scale).to(dtype)
    w = (1 + 0.3 * torch.randn(H, generator=gen)).to(dtype)
    return x.cuda(), w.cuda(), gen


def check_scaled(q, scales, y, rel, what=""):
    """q and scales against the fp64 rows y, each of whose values may be off by rel."""
    q, scales, y = q.double().cpu(), scales.double().cpu(), y.cpu()
    H, blocks = y.shape[1], -(-y.shape[1] // 128)
    assert (scales[:, blocks:] == 0).all(), what
    for b in range(blocks):
        part = y[:, b * 128:(b + 1) * 128]
        fine = torch.where(part.isfinite(), part, 0.0)
        want = fine.abs().amax(1).clamp(min=LEAST) / 448
        got = scales[:, b]
        assert ((got - want).abs() <= (rel + 2 * U) * want).all(), f"{what}: scales of block {b}"
        z = part / got[:, None]
        qb = q[:, b * 128:(b + 1) * 128]
        assert (qb.isnan() == ~part.isfinite()).all(), f"{what}: NaN of block {b}"
        assert (qb.abs().nan_to_num() <= 448).all()
        off = (qb - z).abs().nan_to_num(posinf=0.0)
        step = torch.maximum(z.abs().nan_to_num(posinf=0.0) * 2 ** -4, torch.tensor(2.0 ** -10))
        assert (off <= step + (rel + 4 * U) * z.abs().nan_to_num(posinf=0.0)).all(), \
            f"{what}: values of block {b}"


SIZES = [(1, 8), (3, 64), (5, 520), (2, 1032), (7, 2048), (4, 4096), (3, 4104), (2, 7168),
         (9, 8200), (2, 16384), (1030, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, H, dtype, residual):
    dt = DT[dtype]
    x, w, gen = values(T, H, dt, H + T)
    L = ep.Layout(T, 1, 1, 1, H, 0, dtype=dt)
    out = torch.full_like(x, 7.0)
    res = torch.randn(T, H, generator=gen).mul(3).to(dt).cuda() if residual else None
    s = torch.empty_like(x) if residual else None
    ep.rms_norm(L, x, w, EPS, out=out, residual=res, sum_out=s)
    if residual:
        want = x.double() + res.double()
        assert ((s.double() - want).abs() <= rounded(want, U * want.abs(), dt)).all()
    of = (s if residual else x).double()
    want = of * w.double() / ((of ** 2).mean(1, keepdim=True) + EPS).sqrt()
    assert ((out.double() - want).abs() <= rounded(want, 48 * U * want.abs(), dt)).all()
    if H % 16:
        return
    # in 8 bits beside it, and alone: the same bits each time
    q = torch.empty(T, H, dtype=ep.E4M3, device="cuda")
    sc = torch.full((T, ep.scale_columns(H)), 7.0, device="cuda")
    out2 = torch.empty_like(out)
    ep.rms_norm(L, x, w, EPS, out=out2, out_q=q, out_scales=sc, residual=res, sum_out=s)
    assert torch.equal(out, out2)
    check_scaled(q, sc, want, 48 * U)
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    ep.rms_norm(L, x, w, EPS, out_q=q2, out_scales=sc2, residual=res, sum_out=s)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)


@pytest.mark.parametrize("T,H", [(5, 520), (1030, 264), (4, 4096), (2, 7168), (2, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sum_in_place(T, H, dtype):
    """The residual's buffer, or x's, takes the sum: the same bits as another one."""
    dt = DT[dtype]
    x, w, gen = values(T, H, dt, H + 5)
    res = torch.randn(T, H, generator=gen).to(dt).cuda()
    L = ep.Layout(T, 1, 1, 1, H, 0, dtype=dt)
    out, s, out2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    ep.rms_norm(L, x, w, EPS, out=out, residual=res, sum_out=s)
    for a, b, into in ((x, res.clone(), 1), (x.clone(), res, 0)):
        out2.fill_(7.0)
        total = (a, b)[into]
        ep.rms_norm(L, a, w, EPS, out=out2, residual=b, sum_out=total)
        assert torch.equal(out, out2) and torch.equal(s, total)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_special_rows(dtype):
    """Rows of zeros, tiny and huge rows, an infinity, a NaN: each its own row's
    matter."""
    dt, H = DT[dtype], 400
    x, w, _ = values(7, H, dt, 3)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 40
    x[3, 17] = float("inf")
    x[4, 300] = float("nan")
    x[5, 128:256] = 0
    L = ep.Layout(7, 1, 1, 1, H, 0, dtype=dt)
    out, q = torch.empty_like(x), torch.empty(7, H, dtype=ep.E4M3, device="cuda")
    sc = torch.empty(7, ep.scale_columns(H), device="cuda")
    ep.rms_norm(L, x, w, EPS, out=out, out_q=q, out_scales=sc)
    of = x.double()
    want = of * w.double() / ((of ** 2).mean(1, keepdim=True) + EPS).sqrt()
    for r in (0, 1, 2, 5, 6):
        assert ((out[r].double() - want[r]).abs() <= rounded(want[r], 48 * U * want[r].abs(), dt)).all()
    keep = torch.tensor([0, 1, 2, 5, 6], device="cuda")
    check_scaled(q[keep], sc[keep], want[keep], 48 * U)
    assert (sc[0, :4] == 2.0 ** -100).all() and (q[0].float() == 0).all()
    # 1 / infinity is 0: zeros beside the NaN
    assert out[3, 17].isnan() and (out[3, :17] == 0).all() and q[3, 17].float().isnan()
    assert (q[3, 18:].float() == 0).all()
    assert out[4].isnan().all() and q[4].float().isnan().all() and (sc[4, :4] == 2.0 ** -100).all()


def backward(x, w, g, gs):
    """In 64 bits: the gradients, and the sums of magnitudes that bound them."""
    x, w, g = x.double(), w.double(), g.double()
    r = 1 / ((x ** 2).mean(1, keepdim=True) + EPS).sqrt()
    n, gw = x * r, g * w
    gx = r * (gw - n * (gw * n).mean(1, keepdim=True))
    mag = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    if gs is not None:
        gx, mag = gx + gs.double(), mag + gs.double().abs()
    return gx, mag, (g * n).sum(0), (g * n).abs().sum(0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", SIZES + [(2500, 4096), (4100, 72)])
def test_norm_bwd(T, H, dtype):
    dt = DT[dtype]
    x, w, gen = values(T, H, dt, 5 * H + T)
    g, gs = (torch.randn(T, H, generator=gen).to(dt).cuda() for _ in range(2))
    L = ep.Layout(T, 1, 1, 1, H, 0, dtype=dt)
    ws = ep.new_rms_norm_bwd_workspace(L).fill_(255)
    gx, gw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    ep.rms_norm_bwd(L, g, x, w, EPS, gx, gw, ws, grad_sum=gs)
    want, mag, want_w, mag_w = backward(x, w, g, gs)
    # the dot product's chain as the sum of squares', of terms of both signs: 64 u
    # of their magnitudes, and r's 40 u three times over in n c
    bound = 256 * U * mag
    assert ((gx.double() - want).abs() <= rounded(want, bound, dt)).all()
    # a sum of T terms: a chain of T / partials, then at most 512 partials
    chain = T + 64
    bound_w = (chain + 64) * U * mag_w
    assert ((gw.double() - want_w).abs() <= rounded(want_w, bound_w, dt)).all()
    # without the sum's gradient, and without the weight's (and a workspace); the
    # same bits again
    want, mag, _, _ = backward(x, w, g, None)
    gx1, gx2, gw2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ep.rms_norm_bwd(L, g, x, w, EPS, gx1, gw2, ws)
    assert ((gx1.double() - want).abs() <= rounded(want, 256 * U * mag, dt)).all()
    ep.rms_norm_bwd(L, g, x, w, EPS, gx2)
    assert torch.equal(gx1, gx2) and torch.equal(gw, gw2)


def test_no_rows():
    L = ep.Layout(0, 1, 1, 1, 264, 0, dtype=torch.float32)
    none, w = torch.empty(0, 264, device="cuda"), torch.ones(264, device="cuda")
    gw = torch.full_like(w, 7.0)
    ep.rms_norm(L, none, w, EPS, out=none.clone())
    ep.rms_norm_bwd(L, none, none, w, EPS, none.clone(), gw, ep.new_rms_norm_bwd_workspace(L))
    assert (gw == 0).all()


def test_gradient_against_differences():
    """fp32 rows, so that a difference of 2^-8 stands out of the rounding; the loss
    is linear in the outputs, its second-order part falls out of the central
    difference, and its third-order one is below 2^-16 of the gradient's size."""
    T, H, h = 3, 72, 2.0 ** -8
    x, w, gen = values(T, H, torch.float32, 11)
    res, cy, cs = (torch.randn(T, H, generator=gen).cuda() for _ in range(3))
    leaves = [t.clone().requires_grad_() for t in (x, w, res)]
    y, s = epa.rms_norm(leaves[0], leaves[1], EPS, residual=leaves[2])
    ((y * cy).sum() + (s * cs).sum()).backward()

    def loss(x, w, res):
        s = (x.double() + res.double())
        y = s * w.double() / ((s ** 2).mean(1, keepdim=True) + EPS).sqrt()
        return (y * cy.double()).sum() + (s * cs.double()).sum()

    for i, leaf in enumerate(leaves):
        for at in torch.randint(0, leaf.numel(), (12,), generator=gen).tolist():
            args = [t.detach().double() for t in leaves]
            up, down = [a.clone() for a in args], [a.clone() for a in args]
            up[i].view(-1)[at] += h
            down[i].view(-1)[at] -= h
            want = float(loss(*up) - loss(*down)) / (2 * h)
            got = float(leaf.grad.reshape(-1)[at])
            assert abs(got - want) <= 2.0 ** -12 * max(1.0, abs(want))
