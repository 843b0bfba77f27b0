"""The experts' products and gated activation: cases, plain forms and work.

Between dispatch and combine every expert applies its own weights to the rows
of its segment of the receive buffer. The operators are

  linear      out[r] = W[e] x[r] for the live rows r of expert e (bf16, fp16, fp32)
  linear_bwd  grad_x[r] = W[e]^T grad[r] and grad_w[e] = sum_r grad[r] x[r]^T
  swiglu      out[r] = silu(gate[r]) * up[r], gate and up the halves of a row
  swiglu_bwd  the gradient of both halves
  quant       linear with 4-bit weights, a scale and a zero point per group of inputs

Rows of an expert-major buffer that hold no route (the padding of a segment,
the rows behind the last segment) are zeros in every output.
"""
import math

import torch

#: Set from outside: the framework's kernels instead of the plain forms.
own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _case(name, op, dtype, T, K, E, A, H, N, of=0, route="uniform", group=0, zeros=False):
    """T tokens with K routes each among `of` experts, the first E of them here; segments padded to A rows;
    rows of H values in and N out (swiglu: H values out of 2H in)."""
    return {"name": name, "op": op, "dtype": dtype, "T": T, "K": K, "E": E, "A": A, "H": H, "N": N,
            "of": of or E, "route": route, "group": group, "zeros": zeros}


def listed():
    return [
        # the small workload's layer: where launches and latency count
        _case("linear tiny", "linear", "bf16", 256, 2, 8, 16, 512, 1024),
        # sixteen sequences decoding a token each: about ten rows in a hundred experts, the weights' bytes count
        _case("linear decode", "linear", "bf16", 16, 8, 128, 1, 2048, 1536),
        # a training layer with a hundred experts of uneven load (the first holds many times the last's rows)
        _case("linear zipf", "linear", "bf16", 8192, 8, 128, 128, 2048, 1536, route="zipf"),
        # one GPU's share of an 8-way expert-parallel layer: most routes go elsewhere
        _case("linear share", "linear", "bf16", 32768, 8, 32, 128, 7168, 4096, of=256),
        # odd and ragged sizes in full precision, as a numerics check of a training run has them
        _case("linear_bwd ragged fp32", "linear_bwd", "fp32", 1111, 3, 7, 1, 1032, 776),
        # the second product of a layer with few large experts
        _case("linear_bwd large", "linear_bwd", "bf16", 16384, 2, 8, 128, 14336, 4096),
        # fp16 training with many uneven experts
        _case("linear_bwd zipf fp16", "linear_bwd", "fp16", 8192, 8, 128, 128, 2048, 1536, route="zipf"),
        # the activation between the two products, in the uneven layer and in the layer of few large experts
        _case("swiglu zipf", "swiglu", "bf16", 8192, 8, 128, 128, 768, 0, route="zipf"),
        _case("swiglu_bwd large", "swiglu_bwd", "bf16", 16384, 2, 8, 128, 14336, 0),
        # one sequence decoding with 4-bit weights: the smallest call of serving
        _case("quant one token", "quant", "bf16", 1, 2, 8, 1, 4096, 14336, group=128),
        # a batch decoding with 4-bit weights: about one row each for two thirds of the experts
        _case("quant batch", "quant", "bf16", 32, 8, 256, 1, 7168, 4096, group=128),
        # small groups with zero points, ragged rows, fp16
        _case("quant ragged fp16", "quant", "fp16", 77, 4, 24, 4, 2080, 1000, of=32, group=32, zeros=True),
    ]


def _log(rng, low, high, step=1):
    return max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))) // step * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "swiglu", "swiglu_bwd", "quant", "quant"])
    dtype = rng.choice(["bf16", "bf16", "fp16"] + ([] if op == "quant" else ["fp32"]))
    E = _log(rng, 1, 256)
    of = E * rng.choice([1, 1, 2, 8])
    K = rng.randint(1, min(8, of))
    A = rng.choice([1, 1, 4, 16, 128])
    route = rng.choice(["uniform", "zipf"]) if of == E else "uniform"
    if op == "quant":
        group = rng.choice([32, 64, 128])
        H = max(1, _log(rng, 128, 8192) // group) * group
        N = _log(rng, 128, 8192, 8)
        E = min(E, (1 << 32) // (H * N))
        K = min(K, of)
        return dict(_case("", op, dtype, _log(rng, 1, 128), K, E, A, H, N, max(of, E), route if of == E else "uniform",
                          group, rng.random() < 0.5))
    T = _log(rng, 1, 16384)
    if op.startswith("swiglu"):
        H = _log(rng, 64, 14336, 8)
        T = max(1, min(T, (1 << 27) // (H * K)))
        return dict(_case("", op, dtype, T, K, E, A, H, 0, of, route))
    H, N = _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
    E = max(1, min(E, (1 << 30) // (H * N)))
    cost = (1 << 37) if dtype == "fp32" else (1 << 39)
    T = max(1, min(T, cost // (H * N * K)))
    return dict(_case("", op, dtype, T, K, E, A, H, N, max(of, E), route if of == E else "uniform"))


def _capacity(c):
    """Rows of the receive buffer: enough for every route, or for a quarter more than this share's expected ones."""
    routes = c["T"] * min(c["K"], c["E"])
    if c["of"] > c["E"]:
        routes = min(routes, int(1.25 * c["T"] * c["K"] * c["E"] / c["of"]) + 8 * c["K"])
    return routes + c["E"] * (c["A"] - 1)


def _route(c, gen):
    """Distinct experts for every token, int64 [T, K]; -1 where the expert is not one of the first E."""
    u = torch.rand(c["T"], c["of"], device="cuda", generator=gen, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    score = -torch.log(-torch.log(u))
    if c["route"] == "zipf":
        score = score - 1.1 * torch.log(torch.arange(1, c["of"] + 1, device="cuda", dtype=torch.float64))
    idx = score.topk(c["K"], dim=1).indices
    return torch.where(idx < c["E"], idx, -1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    dtype, E, A, H, N, cap = DTYPES[c["dtype"]], c["E"], c["A"], c["H"], c["N"], _capacity(c)
    idx = _route(c, gen)

    def rows(width):
        return torch.randn(cap, width, device="cuda", generator=gen, dtype=dtype) * live[:, None]

    def weight(scale):
        return torch.randn(E, N, H, device="cuda", generator=gen, dtype=dtype).mul_(scale)

    # the segments: each expert's rows in route order, padded to A; what lies at or past the capacity is dropped
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E).tolist()
    at, segments = 0, []
    for e in range(E):
        n = max(0, min(counts[e], cap - at))
        if n:
            segments.append((e, at, at + n))
        at += -(-counts[e] // A) * A
    live = torch.zeros(cap, device="cuda", dtype=torch.bool)
    for _, a, b in segments:
        live[a:b] = True
    s = {"case": c, "dtype": dtype, "cap": cap, "segments": segments, "live": live.nonzero().squeeze(1)}
    op = c["op"]
    if op in ("linear", "linear_bwd", "quant"):
        s["x"] = rows(H)
    if op in ("linear", "linear_bwd"):
        s["w"] = weight(H ** -0.5)
    if op == "linear_bwd":
        s["grad"] = rows(N)
    if op.startswith("swiglu"):
        s["gate_up"] = rows(2 * H)
    if op == "swiglu_bwd":
        s["grad"] = rows(H)
    if op == "quant":
        groups = H // c["group"]
        s["q"] = torch.randint(0, 256, (E, N, H // 2), device="cuda", generator=gen, dtype=torch.uint8)
        s["scales"] = (torch.rand(E, N, groups, device="cuda", generator=gen) * H ** -0.5 * 0.3 + 1e-3).to(dtype)
        s["zeros"] = (torch.randint(5, 12, (E, N, groups), device="cuda", generator=gen, dtype=torch.uint8)
                      if c["zeros"] else None)
    if own:  # the prepared routing and the output buffers that a program keeps
        import combine_ep_prepare_amd as ep
        s["layout"] = layout = ep.Layout(c["T"], c["K"], E, A, H, cap, dtype=dtype, zero_tail=True)
        s["handle"] = ep.new_handle(layout)
        ep.prepare(layout, idx.contiguous(), torch.empty(E, dtype=torch.int32, device="cuda"), s["handle"])

        def new(*shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        s["out"] = {"linear": lambda: (new(cap, N),), "linear_bwd": lambda: (new(cap, H), new(E, N, H)),
                    "swiglu": lambda: (new(cap, H),), "swiglu_bwd": lambda: (new(cap, 2 * H),),
                    "quant": lambda: (new(cap, N),)}[op]()
    return s


def _run_own(s):
    import combine_ep_prepare_amd as ep
    op, L, h, out = s["case"]["op"], s["layout"], s["handle"], s["out"]
    if op == "linear":
        ep.grouped_linear(L, h, s["x"], s["w"], out[0])
    elif op == "linear_bwd":
        ep.grouped_linear_bwd(L, h, s["grad"], s["x"], s["w"], out[0], out[1])
    elif op == "swiglu":
        ep.swiglu(L, h, s["gate_up"], out[0])
    elif op == "swiglu_bwd":
        ep.swiglu_bwd(L, h, s["grad"], s["gate_up"], out[0])
    else:
        ep.grouped_linear_quant(L, h, s["x"], s["q"], s["scales"], s["zeros"], out[0])
    return list(out)


def _unpacked(q):
    """uint8 [N, H/2] -> fp32 [N, H]: the low four bits are the even column."""
    return torch.stack((q & 15, q >> 4), dim=-1).reshape(q.shape[0], -1).float()


def _scatter(s, values):
    """The values of the live rows in a buffer of zeros, rounded once."""
    out = torch.zeros(s["cap"], values.shape[1], device="cuda", dtype=s["dtype"])
    out[s["live"]] = values.to(s["dtype"])
    return out


def run(state):
    """The plain forms: 32-bit products, one for each expert that has rows (their sizes are ragged), rounded once."""
    s = state
    if own:
        return _run_own(s)
    c, op, dtype = s["case"], s["case"]["op"], s["dtype"]
    if op == "linear":
        out = torch.zeros(s["cap"], c["N"], device="cuda", dtype=dtype)
        for e, a, b in s["segments"]:
            out[a:b] = (s["x"][a:b].float() @ s["w"][e].float().t()).to(dtype)
        return [out]
    if op == "linear_bwd":
        grad_x = torch.zeros(s["cap"], c["H"], device="cuda", dtype=dtype)
        grad_w = torch.zeros(c["E"], c["N"], c["H"], device="cuda", dtype=dtype)
        for e, a, b in s["segments"]:
            g = s["grad"][a:b].float()
            grad_x[a:b] = (g @ s["w"][e].float()).to(dtype)
            grad_w[e] = (g.t() @ s["x"][a:b].float()).to(dtype)
        return [grad_x, grad_w]
    if op == "quant":
        out = torch.zeros(s["cap"], c["N"], device="cuda", dtype=dtype)
        for e, a, b in s["segments"]:
            z = 8.0 if s["zeros"] is None else s["zeros"][e].float()[:, :, None]
            w = _unpacked(s["q"][e]).reshape(c["N"], -1, c["group"])
            w = ((w - z) * s["scales"][e].float()[:, :, None]).reshape(c["N"], -1)
            out[a:b] = (s["x"][a:b].float() @ w.t()).to(dtype)
        return [out]
    gate, up = s["gate_up"][s["live"]].float().chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-gate))
    if op == "swiglu":
        return [_scatter(s, gate * sig * up)]
    grad = s["grad"][s["live"]].float()
    return [_scatter(s, torch.cat((grad * up * sig * (1 + gate * (1 - sig)), grad * gate * sig), dim=1))]


def exact(case, seed):
    """The definition in 64 bits, from the routing's own row lists: out[r] = W[e(r)] x[r] row set by row set."""
    s = prepare(case, seed)
    c, op, cap = case, case["op"], s["cap"]
    expert = torch.full((cap,), -1, device="cuda")
    for e, a, b in s["segments"]:
        expert[a:b] = e
    present = [(e, (expert == e).nonzero().squeeze(1)) for e in sorted({e for e, _, _ in s["segments"]})]
    if op == "linear":
        out = torch.zeros(c["N"], cap, device="cuda", dtype=torch.float64)
        for e, r in present:
            out[:, r] = s["w"][e].double() @ s["x"].index_select(0, r).double().t()
        return [out.t().contiguous()]
    if op == "linear_bwd":
        gx = torch.zeros(c["H"], cap, device="cuda", dtype=torch.float64)
        gw = torch.zeros(c["E"], c["N"], c["H"], device="cuda", dtype=torch.float64)
        for e, r in present:
            gt = s["grad"].index_select(0, r).double().t().contiguous()
            gx[:, r] = s["w"][e].double().t() @ gt
            gw[e] = gt @ s["x"].index_select(0, r).double()
        return [gx.t().contiguous(), gw]
    if op == "quant":
        out = torch.zeros(c["N"], cap, device="cuda", dtype=torch.float64)
        for e, r in present:
            x, q, sc = s["x"].index_select(0, r).double().t(), s["q"][e].int(), s["scales"][e].double()
            z = torch.full_like(sc, 8.0) if s["zeros"] is None else s["zeros"][e].double()
            w = torch.empty(c["N"], c["H"], device="cuda", dtype=torch.float64)
            w[:, 0::2], w[:, 1::2] = (q & 0xF).double(), ((q >> 4) & 0xF).double()
            w = (w - z.repeat_interleave(c["group"], 1)) * sc.repeat_interleave(c["group"], 1)
            out[:, r] = w @ x
        return [out.t().contiguous()]
    H = c["H"]
    g, u = s["gate_up"][:, :H].double(), s["gate_up"][:, H:].double()  # rows without a route hold zeros and give zeros
    sig = torch.sigmoid(g)
    if op == "swiglu":
        return [g * sig * u]
    d = s["grad"].double()
    return [torch.cat((d * u * (sig + g * sig * torch.sigmoid(-g)), d * sig * g), dim=1)]


def _loaded(c):
    """Expected live rows and experts with a row."""
    if c["route"] == "zipf":
        weights = [(e + 1) ** -1.1 for e in range(c["E"])]
        share = [min(1.0, c["K"] * w / sum(weights)) for w in weights]
        return c["T"] * c["K"], sum(1 - (1 - p) ** c["T"] for p in share)
    p = c["K"] / c["of"]
    return c["T"] * c["E"] * p, c["E"] * (1 - (1 - min(1.0, p)) ** c["T"])


def work(case):
    c, op, size = case, case["op"], DTYPES[case["dtype"]].itemsize
    H, N, cap = c["H"], c["N"], _capacity(case)
    R, active = _loaded(c)
    if op == "linear":
        return {"bytes": size * (R * H + active * N * H + cap * N), "flops": 2 * R * H * N}
    if op == "linear_bwd":
        return {"bytes": size * (R * (H + N) + active * N * H + cap * H + c["E"] * N * H), "flops": 4 * R * H * N}
    if op == "quant":
        per = 0.5 + (size + c["zeros"]) / c["group"]
        return {"bytes": size * (R * H + cap * N) + active * N * H * per, "flops": 2 * R * H * N}
    if op == "swiglu":
        return {"bytes": size * (2 * R * H + cap * H), "flops": 6 * R * H}
    return {"bytes": size * (3 * R * H + 2 * cap * H), "flops": 14 * R * H}
