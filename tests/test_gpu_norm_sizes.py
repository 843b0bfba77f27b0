"""The norm at more sizes: backward passes whose blocks take several rows each in every
form of the kernel, rows past the 2^32 threads of one grid, and rows that are not
finite in the backward pass."""
import pytest
import torch

import combine_ep_prepare_amd as ep
import test_gpu_norm as plain
from test_gpu_norm import DT, EPS, U, backward, check_scaled, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# 512 blocks of a row (longer ones) or of four: two or three turns each
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", [(4200, 264), (4200, 520), (4200, 1032), (1100, 2056), (1100, 4104),
                                 (1100, 8200), (1030, 16384)])
def test_several_turns(T, H, dtype):
    plain.test_norm_bwd(T, H, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("H", [72, 520, 4096, 8200])
def test_backward_of_special_rows(H, dtype):
    """An infinity or NaN in x, grad or grad_sum: finite where the formula is, and the
    other rows' bits as without them."""
    dt, T = DT[dtype], 9
    x, w, gen = values(T, H, dt, H)
    w = torch.where(w.abs() < 0.01, torch.ones_like(w), w)
    g, gs = (torch.randn(T, H, generator=gen).to(dt).cuda() for _ in range(2))
    L = ep.Layout(T, 1, 1, 1, H, 0, dtype=dt)
    ws = ep.new_rms_norm_bwd_workspace(L)

    def run():
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        ep.rms_norm_bwd(L, g, x, w, EPS, gx, gw, ws, grad_sum=gs)
        return gx, gw

    clean = run()
    inf = float("inf")
    gs[6, 3], gs[7, H - 1] = inf, float("nan")
    gx, gw = run()
    assert torch.equal(gw, clean[1])
    x[1, 5], g[3, H - 2], g[4, 1] = inf, -inf, float("nan")
    gx, gw = run()
    want, _, want_w, _ = backward(x, w, g, gs)
    assert torch.equal(gx.isfinite(), want.isfinite()) and torch.equal(gw.isfinite(), want_w.isfinite())
    fine = [0, 2, 5, 8]
    assert torch.equal(gx[fine], clean[0][fine])
    keep = want_w.isfinite()
    assert int((~keep).sum()) == 3 and torch.equal(gx[6, 4:], clean[0][6, 4:])
    x[2, 0] = float("nan")
    gx, gw = run()
    assert gx[2].isnan().all() and gw.isnan().all() and torch.equal(gx[[0, 5, 8]], clean[0][[0, 5, 8]])


@pytest.mark.parametrize("H", [16, 64])
def test_rows_past_one_grid(H):
    """A grid has less than 2^32 threads: four rows of 64 lanes a block make 2^26 rows of
    it, and the rest are another's. Rows repeat, so that a few checked ones tell."""
    dt, few = torch.bfloat16, 1021
    T = (1 << 26) + 4 * few + 1
    base, w, gen = values(few, H, dt, H)
    more = torch.randn(few, H, generator=gen).to(dt).cuda()
    at = torch.arange(T, device="cuda") % few

    def outputs(rows):
        return (torch.full((rows, H), 7.0, dtype=dt, device="cuda"),
                torch.full((rows, H), 7.0, dtype=dt, device="cuda"),
                torch.zeros(rows, H, dtype=torch.uint8, device="cuda").view(ep.E4M3),
                torch.full((rows, ep.scale_columns(H)), 7.0, device="cuda"))

    def run(x, residual):
        rows = x.shape[0]
        total, out, q, scales = outputs(rows)
        ep.rms_norm(ep.Layout(rows, 1, 1, 1, H, 0, dtype=dt), x, w, EPS, out=out, out_q=q,
                    out_scales=scales, residual=residual, sum_out=total)
        return total, out, q.view(torch.uint8), scales

    small = run(base, more)
    of = small[0].double()
    want = of * w.double() / ((of ** 2).mean(1, keepdim=True) + EPS).sqrt()
    assert ((small[1].double() - want).abs() <= plain.rounded(want, 48 * U * want.abs(), dt)).all()
    check_scaled(small[2].view(ep.E4M3), small[3], want, 48 * U)
    large = run(base[at], more[at])
    part = 1 << 22
    for a in range(0, T, part):
        for got, ref in zip(large, small):
            assert torch.equal(got[a:a + part], ref[at[a:a + part]]), a
