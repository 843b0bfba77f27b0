"""The experts' ops at the ends of what their documentation allows."""
import pytest
import torch

import combine_ep_prepare_amd as ep

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
