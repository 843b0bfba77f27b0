"""The experts' layer in 8 bits, its norm, and the whole layer for a few tokens: cases, plain forms and work.

A layer in 8 bits runs from the norm in front of it to the combine behind it on
rows of e4m3 values with one fp32 scale for every 128 of a row, and weights of
e4m3 values with one for every 128 x 128. The operators are

  norm      s = x + residual, y = s / rms(s) * weight; y in the payload type or in 8 bits with scales
  norm_bwd  the gradients of s and of weight
  linear    out[r] = W[e] x[r] for the live rows r of expert e, both in 8 bits
  act       silu(gate[r]) * up[r] in 8 bits with scales, gate and up the halves of a row
  layer     sum over a token's routes k of w[k] * W_down[e] (silu(W_gate[e] x) * W_up[e] x), without a
            prepared routing; weights in the payload type or in 8 bits

Rows of an expert-major buffer that hold no route are zeros in every output.
"""
import math

import torch

#: Set from outside: the framework's kernels instead of the plain forms.
own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK, TOP, LEAST = 128, 448.0, 448.0 * 2.0 ** -100   # of a scale: values, the type's largest, the least amax
EPS = 1e-6


def _norm(name, op, dtype, T, H, residual=True, quant=False):
    """T rows of H values; with a residual that is added (norm_bwd: a gradient that comes in on the sum)."""
    return {"name": name, "op": op, "dtype": dtype, "T": T, "H": H, "residual": residual, "quant": quant}


def _expert(name, op, dtype, T, K, E, A, H, N, of=0, route="uniform", quant=True):
    """T tokens with K routes each among `of` experts, the first E of them here; segments padded to A rows.
    linear: rows of H values in and N out; act: H values out of 2H in; layer: rows of H, N between the products."""
    return {"name": name, "op": op, "dtype": dtype, "T": T, "K": K, "E": E, "A": A, "H": H, "N": N,
            "of": of or E, "route": route, "quant": quant}


def listed():
    return [
        # sixteen sequences decoding a token each: the norm in front of the layer, where launches count
        _norm("norm decode", "norm", "bf16", 16, 7168, quant=True),
        # a prompt's norm in front of an 8-bit dispatch
        _norm("norm large", "norm", "bf16", 32768, 7168, quant=True),
        # odd sizes in full precision, as a numerics check of a training run has them
        _norm("norm_bwd ragged fp32", "norm_bwd", "fp32", 1111, 1032, residual=False),
        # a training step of a layer with few large experts
        _norm("norm_bwd large", "norm_bwd", "bf16", 16384, 4096),
        # a batch decoding in 8 bits: about one row each for two thirds of the experts, the weights' bytes count
        _expert("linear decode", "linear", "bf16", 32, 8, 256, 1, 7168, 4096),
        # the first product of a prompt in a layer with few large experts
        _expert("linear large", "linear", "bf16", 16384, 2, 8, 128, 4096, 28672),
        # ragged rows and features, a last block that is not full, fp16 out
        _expert("linear ragged fp16", "linear", "fp16", 1111, 3, 7, 1, 1040, 776),
        # the activation of a layer with a hundred experts of uneven load, and of one with few large experts
        _expert("act zipf", "act", "bf16", 8192, 8, 128, 128, 768, 0, route="zipf"),
        _expert("act large", "act", "bf16", 16384, 2, 8, 128, 14336, 0),
        # one sequence decoding: two large experts in 16 bits
        _expert("layer token", "layer", "bf16", 1, 2, 8, 1, 4096, 14336, quant=False),
        # a batch decoding in 8 bits: a hundred of many experts, about one row each
        _expert("layer batch", "layer", "bf16", 16, 8, 256, 1, 7168, 2048),
        # the smallest call: a few tokens, half their routes elsewhere, odd sizes, fp16
        _expert("layer ragged fp16", "layer", "fp16", 5, 3, 7, 1, 1032, 776, of=14, quant=False),
    ]


def _log(rng, low, high, step=1):
    return max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "linear", "linear", "act", "layer", "layer", "layer"])
    if op.startswith("norm"):
        quant = op == "norm" and rng.random() < 0.6
        H = _log(rng, 64, 16384, 16 if quant else 8)
        T = min(_log(rng, 1, 32768), (1 << 27) // H)
        return dict(_norm("", op, rng.choice(["bf16", "bf16", "fp16", "fp32"]), T, H, rng.random() < 0.7, quant))
    dtype = rng.choice(["bf16", "bf16", "fp16"] + (["fp32"] if op == "act" else []))
    E = _log(rng, 1, 256)
    of = E * rng.choice([1, 1, 2, 8])
    K = rng.randint(1, min(8, of))
    A = rng.choice([1, 1, 4, 16, 128])
    if op == "layer":
        quant = rng.random() < 0.5
        H, I = _log(rng, 64, 8192, 16 if quant else 8), _log(rng, 64, 14336, 16 if quant else 8)
        E = max(1, min(E, (1 << 32) // (3 * H * I)))
        return dict(_expert("", op, dtype, _log(rng, 1, 64), K, E, 1, H, I, max(of, E), quant=quant))
    route = rng.choice(["uniform", "zipf"]) if of == E else "uniform"
    T = _log(rng, 1, 16384)
    if op == "act":
        H = _log(rng, 64, 14336, 16)
        T = max(1, min(T, (1 << 27) // (H * K)))
        return dict(_expert("", op, dtype, T, K, E, A, H, 0, of, route))
    H, N = _log(rng, 64, 8192, 16), _log(rng, 64, 8192, 8)
    E = max(1, min(E, (1 << 31) // (H * N)))
    T = max(1, min(T, (1 << 40) // (H * N * K)))
    return dict(_expert("", op, dtype, T, K, E, A, H, N, max(of, E), route if of == E else "uniform"))


def _capacity(c):
    """Rows of the receive buffer: enough for every route, or for a quarter more than this share's expected ones."""
    routes = c["T"] * min(c["K"], c["E"])
    if c["of"] > c["E"]:
        routes = min(routes, int(1.25 * c["T"] * c["K"] * c["E"] / c["of"]) + 8 * c["K"])
    return routes + c["E"] * (c["A"] - 1)


def _blocks(n):
    return -(-n // BLOCK)


def _columns(n):
    """Scales that a row of n values has room for: whole groups of eight."""
    return -(-n // (8 * BLOCK)) * 8


def _route(c, gen):
    """Distinct experts for every token, int64 [T, K]; -1 where the expert is not one of the first E."""
    u = torch.rand(c["T"], c["of"], device="cuda", generator=gen, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    score = -torch.log(-torch.log(u))
    if c["route"] == "zipf":
        score = score - 1.1 * torch.log(torch.arange(1, c["of"] + 1, device="cuda", dtype=torch.float64))
    idx = score.topk(c["K"], dim=1).indices
    return torch.where(idx < c["E"], idx, -1).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    op, dtype, T, H = c["op"], DTYPES[c["dtype"]], c["T"], c["H"]
    s = {"case": c, "dtype": dtype}

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=dtype)

    if op.startswith("norm"):
        s["x"] = normal(T, H)
        s["residual"] = normal(T, H) * 4 if c["residual"] and op == "norm" else None
        s["weight"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype)
        if op == "norm_bwd":
            s["grad"] = normal(T, H)
            s["grad_sum"] = normal(T, H) if c["residual"] else None
        if own:
            _keep_norm(s)
        return s
    E, N, cap = c["E"], c["N"], _capacity(c)
    s["idx"] = idx = _route(c, gen)

    def weights(rows, cols):
        """[E, rows, cols] in the payload type, or e4m3 values and their scales."""
        if not c["quant"]:
            return normal(E, rows, cols).mul_(cols ** -0.5), None
        q = torch.empty(E, rows, cols, device="cuda", dtype=E4M3)
        for e in range(E):
            q[e] = (torch.randn(rows, cols, device="cuda", generator=gen) * 96).clamp_(-TOP, TOP).to(E4M3)
        scales = torch.rand(E, _blocks(rows), _blocks(cols), device="cuda", generator=gen)
        return q, (scales + 0.5) * (cols ** -0.5 / 96)

    if op == "layer":
        flat = idx.reshape(-1)
        s["x"], s["w"] = normal(T, H), torch.rand(T, c["K"], device="cuda", generator=gen) + 0.05
        s["w"] /= s["w"].sum(1, keepdim=True)
        s["gate_up"], s["down"] = weights(2 * N, H), weights(H, N)
        s["routes"] = [(e, (flat == e).nonzero().squeeze(1)) for e in sorted(set(flat[flat >= 0].tolist()))]
        if own:
            import combine_ep_prepare_amd as ep
            s["layout"] = layout = ep.Layout(T, c["K"], E, 1, H, 0, dtype=dtype)
            s["workspace"] = ep.new_expert_layer_workspace(layout, N)
            s["out"] = torch.empty(T, H, device="cuda", dtype=dtype)
        return s
    # the segments: each expert's rows in route order, padded to A; what lies at or past the capacity is dropped
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E).tolist()
    at, segments = 0, []
    for e in range(E):
        n = max(0, min(counts[e], cap - at))
        if n:
            segments.append((e, at, at + n))
        at += -(-counts[e] // c["A"]) * c["A"]
    live = torch.zeros(cap, device="cuda", dtype=torch.bool)
    for _, a, b in segments:
        live[a:b] = True
    s |= {"cap": cap, "segments": segments, "live": live.nonzero().squeeze(1)}
    if op == "act":
        s["gate_up"] = normal(cap, 2 * H) * live[:, None]
    else:
        q = torch.randn(cap, H, device="cuda", generator=gen).mul_(100).clamp_(-TOP, TOP)
        s["x"] = (q * live[:, None]).to(E4M3)
        scales = (torch.rand(cap, _columns(H), device="cuda", generator=gen) * 1.5 + 0.5) / 100
        scales[:, _blocks(H):] = 0
        s["x_scales"] = scales * live[:, None]
        s["w"] = weights(N, H)
    if own:  # the prepared routing and the output buffers that a program keeps
        import combine_ep_prepare_amd as ep
        s["layout"] = layout = ep.Layout(T, c["K"], E, c["A"], H, cap, dtype=dtype, zero_tail=True)
        s["handle"] = ep.new_handle(layout)
        ep.prepare(layout, idx, torch.empty(E, dtype=torch.int32, device="cuda"), s["handle"])
        s["out"] = ([torch.empty(cap, N, device="cuda", dtype=dtype)] if op == "linear" else
                    [torch.empty(cap, H, device="cuda", dtype=E4M3),
                     torch.empty(cap, _columns(H), device="cuda")])
    return s


def _keep_norm(s):
    import combine_ep_prepare_amd as ep
    c, x = s["case"], s["x"]
    s["layout"] = layout = ep.Layout(c["T"], 1, 1, 1, c["H"], 0, dtype=s["dtype"])
    if c["op"] == "norm_bwd":
        s["workspace"] = ep.new_rms_norm_bwd_workspace(layout)
        s["out"] = [torch.empty_like(x), torch.empty_like(s["weight"])]
        return
    s["sum"] = torch.empty_like(x) if c["residual"] else None
    s["out"] = ([torch.empty_like(x, dtype=E4M3), torch.empty(c["T"], _columns(c["H"]), device="cuda")]
                if c["quant"] else [torch.empty_like(x)])


def _run_own(s):
    import combine_ep_prepare_amd as ep
    c, L, out = s["case"], s["layout"], s["out"]
    op = c["op"]
    if op == "norm":
        q, scales = out if c["quant"] else (None, None)
        ep.rms_norm(L, s["x"], s["weight"], EPS, out=None if c["quant"] else out[0], out_q=q, out_scales=scales,
                    residual=s["residual"], sum_out=s["sum"])
        return ([s["sum"]] if c["residual"] else []) + out
    if op == "norm_bwd":
        ep.rms_norm_bwd(L, s["grad"], s["x"], s["weight"], EPS, out[0], out[1], s["workspace"],
                        grad_sum=s["grad_sum"])
    elif op == "linear":
        ep.grouped_linear_scaled(L, s["handle"], s["x"], s["x_scales"], *s["w"], out[0])
    elif op == "act":
        ep.swiglu_scaled(L, s["handle"], s["gate_up"], out[0], out[1])
    else:
        ep.expert_layer(L, s["idx"], s["w"], s["x"], s["gate_up"][0], s["down"][0], out, s["workspace"],
                        gate_up_scales=s["gate_up"][1], down_scales=s["down"][1])
        return [out]
    return list(out)


def _in_blocks(y):
    """Rows of any length cut into blocks of 128, the last one filled up with zeros."""
    n = _blocks(y.shape[1]) * BLOCK
    return torch.nn.functional.pad(y, (0, n - y.shape[1])).view(y.shape[0], -1, BLOCK)


def _to_8_bits(y):
    """e4m3 values and fp32 scales [rows, _columns] of fp32 rows."""
    b = _in_blocks(y)
    scale = b.abs().amax(2).clamp_min(LEAST) / TOP
    q = (b / scale[:, :, None]).view(y.shape[0], -1)[:, :y.shape[1]].to(E4M3)
    return [q.contiguous(), torch.nn.functional.pad(scale, (0, _columns(y.shape[1]) - scale.shape[1]))]


def _wide(q, scales):
    """fp32 values of weights [rows, cols]: e4m3 with scales by 128 x 128, or the payload type without."""
    if scales is None:
        return q.float()
    scales = scales.repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * scales


def _scatter(s, values):
    """The values of the live rows in a buffer of zeros."""
    out = torch.zeros(s["cap"], values.shape[1], device="cuda", dtype=values.dtype)
    if values.dtype == E4M3:
        out.view(torch.uint8)[s["live"]] = values.view(torch.uint8)
    else:
        out[s["live"]] = values
    return out


def run(state):
    """The plain forms: 32 bits, rounded once; products one for each expert that has rows (their sizes are ragged)."""
    s = state
    if own:
        return _run_own(s)
    c, dtype = s["case"], s["dtype"]
    op = c["op"]
    if op == "norm":
        x, more = s["x"], []
        if c["residual"]:
            x = (x.float() + s["residual"].float()).to(dtype)   # the sum is an output, and the norm is that of it
            more = [x]
        x = x.float()
        y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * s["weight"].float()
        return more + (_to_8_bits(y) if c["quant"] else [y.to(dtype)])
    if op == "norm_bwd":
        x, g = s["x"].float(), s["grad"].float()
        r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        n, gw = x * r, g * s["weight"].float()
        grad = r * (gw - n * (gw * n).mean(1, keepdim=True))
        if c["residual"]:
            grad = grad + s["grad_sum"].float()
        return [grad.to(dtype), (g * n).sum(0).to(dtype)]
    if op == "act":
        gate, up = s["gate_up"][s["live"]].float().chunk(2, dim=1)
        q, scales = _to_8_bits(gate / (1 + torch.exp(-gate)) * up)
        return [_scatter(s, q), _scatter(s, scales)]
    if op == "linear":
        out = torch.zeros(s["cap"], c["N"], device="cuda", dtype=dtype)
        x = s["x"].float() * s["x_scales"].repeat_interleave(BLOCK, 1)[:, :c["H"]]
        for e, a, b in s["segments"]:
            out[a:b] = (x[a:b] @ _wide(s["w"][0][e], None if s["w"][1] is None else s["w"][1][e]).t()).to(dtype)
        return [out]
    y = torch.zeros(c["T"] * c["K"], c["H"], device="cuda")
    (gu, gus), (dn, dns) = s["gate_up"], s["down"]
    for e, r in s["routes"]:
        gate, up = (s["x"][r // c["K"]].float() @ _wide(gu[e], None if gus is None else gus[e]).t()).chunk(2, dim=1)
        y[r] = (gate / (1 + torch.exp(-gate)) * up) @ _wide(dn[e], None if dns is None else dns[e]).t()
    return [(y.view(c["T"], c["K"], -1) * s["w"][:, :, None]).sum(1).to(dtype)]


def _exact_8_bits(y):
    """What the e4m3 values are rounded from, and the scales, of rows in 64 bits."""
    scales = torch.zeros(y.shape[0], _columns(y.shape[1]), device="cuda", dtype=torch.float64)
    out = torch.empty_like(y)
    for b in range(_blocks(y.shape[1])):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        scales[:, b] = torch.maximum(part.max(1).values, -part.min(1).values).clamp(min=LEAST) / TOP
        out[:, b * BLOCK:(b + 1) * BLOCK] = part / scales[:, b:b + 1]
    return [out, scales]


def exact(case, seed):
    """The definitions in 64 bits; values in 8 bits as they are before their rounding."""
    s = prepare(case, seed)
    c, op, dtype = case, case["op"], s["dtype"]

    def matrix(pair, e):
        q, scales = pair
        w = q[e].double()
        if scales is not None:
            for i in range(scales.shape[1]):
                w[i * BLOCK:(i + 1) * BLOCK] *= scales[e, i].double().repeat_interleave(BLOCK)[:w.shape[1]]
        return w

    if op.startswith("norm"):
        x, first = s["x"].double(), []
        if op == "norm" and c["residual"]:
            first = [x + s["residual"].double()]
            x = first[0].to(dtype).double()
        rms = ((x ** 2).sum(1, keepdim=True) / c["H"] + EPS) ** 0.5
        if op == "norm":
            y = x * s["weight"].double() / rms
            return first + (_exact_8_bits(y) if c["quant"] else [y])
        g, w = s["grad"].double(), s["weight"].double()
        grad = g * w / rms - x * ((g * w * x).sum(1, keepdim=True) / (c["H"] * rms ** 3))
        if c["residual"]:
            grad += s["grad_sum"].double()
        return [grad, torch.mv((x / rms * g).t(), torch.ones(c["T"], device="cuda", dtype=torch.float64))]
    if op == "act":
        g, u = s["gate_up"][:, :c["H"]].double(), s["gate_up"][:, c["H"]:].double()
        q, scales = _exact_8_bits(g * torch.sigmoid(g) * u)
        dead = torch.ones(s["cap"], device="cuda", dtype=torch.bool)
        dead[s["live"]] = False
        scales[dead] = 0   # rows without a route hold zeros, their scales too
        return [q, scales]
    if op == "linear":
        out = torch.zeros(s["cap"], c["N"], device="cuda", dtype=torch.float64)
        for e, a, b in s["segments"]:
            x = s["x"][a:b].double()
            for i in range(_blocks(c["H"])):
                x[:, i * BLOCK:(i + 1) * BLOCK] *= s["x_scales"][a:b, i:i + 1].double()
            out[a:b] = (matrix(s["w"], e) @ x.t()).t()
        return [out]
    out = torch.zeros(c["T"], c["H"], device="cuda", dtype=torch.float64)
    for e, r in s["routes"]:
        gu = matrix(s["gate_up"], e) @ s["x"].index_select(0, r // c["K"]).double().t()
        g, u = gu[:c["N"]], gu[c["N"]:]
        y = matrix(s["down"], e) @ (g * torch.sigmoid(g) * u)
        out.index_add_(0, r // c["K"], (y * s["w"].reshape(-1)[r].double()).t().contiguous())
    return [out]


def _loaded(c):
    """Expected live rows and experts with a row."""
    if c["route"] == "zipf":
        weights = [(e + 1) ** -1.1 for e in range(c["E"])]
        share = [min(1.0, c["K"] * w / sum(weights)) for w in weights]
        return c["T"] * c["K"], sum(1 - (1 - p) ** c["T"] for p in share)
    p = c["K"] / c["of"]
    return c["T"] * c["E"] * p, c["E"] * (1 - (1 - min(1.0, p)) ** c["T"])


def work(case):
    c, op, size, T, H = case, case["op"], DTYPES[case["dtype"]].itemsize, case["T"], case["H"]
    row8 = H + 4 * _columns(H)   # bytes of a row in 8 bits
    if op == "norm":
        moved = size * (3 if c["residual"] else 1) * H + (row8 if c["quant"] else size * H)
        return {"bytes": T * moved + size * H, "flops": 8 * T * H}
    if op == "norm_bwd":
        return {"bytes": size * H * (T * (4 if c["residual"] else 3) + 2), "flops": 14 * T * H}
    R, active = _loaded(c)
    N = c["N"]
    per = 1 + 4 / BLOCK ** 2 if c["quant"] else size   # bytes of a weight
    if op == "linear":
        return {"bytes": R * row8 + active * N * H * per + size * _capacity(c) * N, "flops": 2 * R * H * N}
    if op == "act":
        return {"bytes": 2 * size * R * H + _capacity(c) * row8, "flops": 8 * R * H}
    return {"bytes": active * 3 * N * H * per + T * (2 * size * H + 12 * c["K"]), "flops": 6 * R * H * N}
