"""The 8-bit product with few rows an expert: sums held in fp32, also of products whose
sizes lie far apart.

Operands take every finite e4m3 value alike, so that a block's products reach from
2^-18 to 2^17 in magnitude. Off by at most n steps of 2^-23 of the sum of the terms'
magnitudes for n terms, and 4 steps more a block, as a product of 16-bit operands is.
Of whole numbers whose sums stay below 2^24 nothing is lost at all, a 1 beside 2^16
included.
"""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_experts import Case, sum_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def any_bits(gen, *shape):
    bits = torch.randint(0, 127, shape, generator=gen) | torch.randint(0, 2, shape, generator=gen) << 7
    return bits.to(torch.uint8).view(ep.E4M3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,E,H,N", [(1, 1, 1, 16, 8), (1, 8, 8, 1152, 136), (12, 2, 6, 272, 264),
                                       (32, 1, 1, 2064, 72), (40, 3, 40, 640, 1032)])
def test_few_rows(T, K, E, H, N, dtype):
    c = Case("any", T, K, E, 1, dtype, seed=T + N)
    x, w = any_bits(c.gen, c.cap, H), any_bits(c.gen, E, N, H)
    xs = torch.full((c.cap, ep.scale_columns(H)), 2.0 ** -9)
    ws = torch.full((E, -(-N // 128), -(-H // 128)), 2.0 ** -9)
    out = c.out(c.cap, N)
    ep.grouped_linear_scaled(c.layout(H), c.handle, x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out)
    want, bound = (torch.zeros(c.cap, N, dtype=torch.float64) for _ in range(2))
    for e, (a, b) in enumerate(c.rows):
        xv, wv = x[a:b].double() * 2.0 ** -9, w[e].double() * 2.0 ** -9
        want[a:b] = xv @ wv.t()
        bound[a:b] = sum_bound(H + 4 * (-(-H // 128)), xv.abs() @ wv.abs().t())
    c.check_rows(out, want, bound, f"H={H} N={N}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,E,H,N", [(1, 1, 1, 16, 8), (12, 2, 6, 272, 264), (32, 1, 1, 1040, 72)])
def test_ones_beside_large_products(T, K, E, H, N, dtype):
    """Two products of 2^16 in every eight, which cancel, and six of -1, 0 or 1."""
    c = Case("any", T, K, E, 1, dtype, seed=T + N)
    x = torch.randint(-1, 2, (c.cap, H), generator=c.gen).float()
    w = torch.randint(-1, 2, (E, N, H), generator=c.gen).float()
    x[:, 0::8] = x[:, 1::8] = 256
    w[:, :, 0::8], w[:, :, 1::8] = 256, -256
    xs = torch.ones(c.cap, ep.scale_columns(H))
    ws = torch.ones(E, -(-N // 128), -(-H // 128))
    out = c.out(c.cap, N)
    ep.grouped_linear_scaled(c.layout(H), c.handle, x.to(ep.E4M3).cuda(), xs.cuda(),
                             w.to(ep.E4M3).cuda(), ws.cuda(), out)
    want = torch.zeros(c.cap, N, dtype=torch.float64)
    for e, (a, b) in enumerate(c.rows):
        want[a:b] = x[a:b].double() @ w[e].double().t()
    assert float(want.abs().max()) <= 256    # whole numbers of every type
    c.check_rows(out, want, torch.zeros_like(want), f"H={H} N={N}")
