"""The activation in 8 bits where single values of a block are not finite, and with large
gates.

A value that is not finite becomes NaN in its own place; its neighbours' scale is that of
the finite ones and they are rounded as ever. The gate's exponent is rounded, which
takes the activation off by up to 2 |g| units of 2^-24 more than its 24 (see
test_gpu_layer); a gate below -174 gives 0 where the definition has less than 2^-250.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_experts import Case
from test_gpu_norm import U, check_scaled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(c, inner, gu, gates=0.0):
    L = c.layout(inner)
    q = torch.full((c.cap, inner), 7.0, device="cuda").to(ep.E4M3)
    s = torch.full((c.cap, ep.scale_columns(inner)), 7.0, device="cuda")
    ep.swiglu_scaled(L, c.handle, gu.cuda(), q, s)
    g, u = gu.double().chunk(2, 1)
    check_scaled(q.cpu()[c.live], s.cpu()[c.live], (g * torch.sigmoid(g) * u)[c.live],
                 (24 + 2 * gates) * U)
    return q.cpu(), s.cpu()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inner", [16, 208, 400])
def test_single_values(inner, dtype):
    """Infinities and NaN in the first and last place of a block, two in one block, in
    the last block that is not full, and over a whole block."""
    c = Case("masked", 40, 4, 8, 4, dtype, seed=inner)
    inf, nan = float("inf"), float("nan")
    gu = c.buffer(2 * inner)
    clean = run(c, inner, gu)
    rows = c.live.nonzero()[:, 0].tolist()
    assert len(rows) > 12
    gate, up, last = 0, inner, inner - 1
    top = min(127, last)
    for row, places in zip(rows[::2], [
            [(gate, inf)], [(gate, -inf)], [(up, inf)], [(up + top, -inf)], [(gate + top, nan)],
            [(up + last, nan)], [(gate + last, inf), (up + last // 2, nan)],
            [(gate + 3, inf), (gate + 9, -inf)], [(up + last, -inf), (gate + last, nan)]]):
        for at, v in places:
            gu[row, at] = v
    gu[rows[18], :top + 1] = nan                       # a whole block
    q, s = run(c, inner, gu)
    untouched = [r for i, r in enumerate(rows) if i % 2 or i > 18]
    assert torch.equal(q[untouched].view(torch.uint8), clean[0][untouched].view(torch.uint8))
    assert torch.equal(s[untouched], clean[1][untouched])
    assert float(s[rows[18], 0]) == 2.0 ** -100


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scale", [4.0, 60.0])
def test_large_gates(scale, dtype):
    c = Case("any", 60, 3, 7, 16, dtype, seed=6)
    gu = c.buffer(2 * 272, scale)
    run(c, 272, gu, float(gu[c.live].abs().max()))
