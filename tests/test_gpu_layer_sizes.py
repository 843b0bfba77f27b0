"""The layer for a few tokens with 8-bit weights where its second product's tiles of 64
columns end inside a tile, and with weights past 2^31 elements."""
import pytest
import torch

import combine_ep_prepare_amd as ep
from test_gpu_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind,T,K,E,H,I", [
    ("any", 64, 8, 128, 272, 144), ("any", 64, 8, 128, 208, 80), ("masked", 64, 8, 256, 1056, 48),
    ("any", 64, 8, 128, 240, 144), ("steep", 64, 16, 128, 368, 272), ("repeat", 128, 8, 160, 176, 16)])
def test_tiles_of_64_columns(kind, T, K, E, H, I, dtype):
    # tiles of the most experts that the routes can reach fill the CUs; smaller grids
    # take tiles of 32
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert H % 64 != 0 and min(T * K, E) * -(-H // 64) >= cus
    case = Layer(kind, T, K, E, H, I, dtype, True)
    out = case.run()
    case.check(out)
    assert torch.equal(case.run(), out)


@pytest.mark.parametrize("eight", [False, True])
def test_weights_past_31_bits(eight):
    """80 experts of 7168 x 4096, 4.7e9 and 2.3e9 weights: the same bits as from three
    experts alone. The other experts' weights are NaN."""
    E, H, I, T, K = 80, 7168, 4096, 5, 2
    used = (1, 37, 79)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dt = ep.E4M3 if eight else torch.bfloat16

    def weights(rows, cols):
        few = torch.randn(3, rows, cols, device="cuda", generator=gen)
        few = (few * 90).clamp_(-448, 448).to(dt) if eight else few.mul_(cols ** -0.5).to(dt)
        all_ = torch.empty(E, rows, cols, dtype=dt, device="cuda")
        all_.view(torch.uint8).fill_(0xFF)       # NaN of either type
        scales = few_scales = None
        if eight:
            few_scales = (torch.rand(3, rows // 128, cols // 128, device="cuda", generator=gen)
                          + 0.5) * (cols ** -0.5 / 90)
            scales = torch.full((E, rows // 128, cols // 128), float("nan"), device="cuda")
        for i, e in enumerate(used):
            all_[e] = few[i]
            if eight:
                scales[e] = few_scales[i]
        assert all_.numel() > 1 << 31
        return few, few_scales, all_, scales

    w1, w2 = weights(2 * I, H), weights(H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    tw = torch.rand(T, K, device="cuda", generator=gen)
    few_idx = torch.tensor([[0, 1], [2, 0], [1, 2], [2, -1], [-1, 1]], device="cuda")
    idx = torch.where(few_idx >= 0, torch.tensor(used, device="cuda")[few_idx.clamp(min=0)], -1)

    def run(experts, idx, gu, gus, dn, dns):
        L = ep.Layout(T, K, experts, 1, H, 0, dtype=torch.bfloat16)
        out = torch.full_like(x, 7.0)
        ep.expert_layer(L, idx, tw, x, gu, dn, out, ep.new_expert_layer_workspace(L, I), gus, dns)
        return out

    want = run(3, few_idx, w1[0], w1[1], w2[0], w2[1])
    got = run(E, idx, w1[2], w1[3], w2[2], w2[3])
    assert want.isfinite().all() and float(want.abs().max()) > 0 and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("eight", [False, True])
def test_two_graphs_share_a_workspace(eight, dtype):
    """Captured calls of two sizes with one workspace, replayed in turn, on rows and
    routes that change between replays."""
    a = Layer("masked", 6, 3, 7, 272, 208, dtype, eight, seed=1)
    b = Layer("any", 3, 5, 9, 144, 400, dtype, eight, seed=2)
    if a.workspace.numel() < b.workspace.numel():
        a.workspace = b.workspace
    b.workspace = a.workspace
    graphs, outs = [], []
    for case in (a, b):
        case.run()
        out = torch.zeros_like(case.x, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            case.run(out)
        graphs.append(graph)
        outs.append(out)
    gen = torch.Generator().manual_seed(5)
    for _ in range(3):
        for case, graph, out in zip((a, b), graphs, outs):
            case.x = (torch.randn(case.x.shape, generator=gen) * 8).to(case.dt)
            case.idx = case.idx[torch.randperm(case.idx.shape[0], generator=gen)].contiguous()
            case.args[2].copy_(case.x)
            case.args[0].copy_(case.idx)
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            case.check(out)
