"""The grouped products of a mixture-of-experts feed-forward block, as cases to measure.

Rows that belong to one expert stand together (the order that the layer's regroup leaves): group e owns rows
offsets[e] .. offsets[e + 1] - 1, and one call covers all groups.

  quantize       codes[r, :] = rint(x[r, :] 127 / a_r), scale[r] = a_r / 127, a_r = max |x[r, :]|
  int8_product   y[r, n] = scale[r] w_scale[e, n] sum_k codes[r, k] w[e, n, k]
  int8_gated     h[r, f] = act(G[r, f]) U[r, f], G and U the int8 products with rows f and F + f of w[e]
  product        y = x w[e]^T; backward: dx = dy w[e], dw[e] = dy_e^T x_e
  gated          h = act(G) U, (G, U) = x w[e]^T, which are also returned for the backward pass where a step trains;
                 backward: dG = dh U act'(G), dU = dh act(G), dx = (dG, dU) w[e], dw[e] = (dG, dU)_e^T x_e

With `own` false, `run` computes them in elementary torch operations in 32 bits (the codes, whose rounding decides
between two whole numbers, in 64); with `own` true it calls the framework's kernels.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's hidden states (16 tokens), quantised for the experts' products
        {"name": "quantize decode", "op": "quantize", "rows": 16, "k": 4096, "type": "bf16"},
        # the inner activations of a 4096-token, top-2 prefill chunk, quantised for the down product
        {"name": "quantize prefill", "op": "quantize", "rows": 8192, "k": 14336, "type": "bf16"},
        # one token through one fine-grained expert's down projection: the smallest call, latency counts
        {"name": "int8 product one row", "op": "int8_product", "rows": 1, "n": 4096, "k": 2048, "groups": 1,
         "skew": 0.0, "type": "bf16"},
        # the down projection of a 2048-token, top-2 prefill chunk over 8 experts
        {"name": "int8 product prefill", "op": "int8_product", "rows": 4096, "n": 4096, "k": 14336, "groups": 8,
         "skew": 0.5, "type": "bf16"},
        # gate/up of a 16-token, top-2 decode step over 8 experts: bound by the weights' bytes
        {"name": "int8 gated decode", "op": "int8_gated", "rows": 32, "n": 14336, "k": 4096, "groups": 8,
         "skew": 0.5, "act": "silu", "type": "bf16"},
        # gate/up of a 4096-token, top-6 prefill chunk over 64 fine-grained experts, unevenly routed
        {"name": "int8 gated fine prefill", "op": "int8_gated", "rows": 24576, "n": 2048, "k": 4096, "groups": 64,
         "skew": 1.0, "act": "silu", "type": "fp16"},
        # a short batch through a narrow block of odd widths
        {"name": "product odd", "op": "product", "rows": 77, "n": 1000, "k": 1416, "groups": 3, "skew": 0.8,
         "type": "fp16"},
        # the 16-bit down projection of a 2048-token, top-2 chunk over 8 experts
        {"name": "product prefill", "op": "product", "rows": 4096, "n": 4096, "k": 14336, "groups": 8, "skew": 0.5,
         "type": "bf16"},
        # its gradients where 64 fine-grained experts train: short ragged groups, many weight gradients
        {"name": "product backward fine", "op": "product_backward", "rows": 24576, "n": 4096, "k": 2048, "groups": 64,
         "skew": 1.0, "type": "bf16"},
        # a 16-token decode step through one shared expert
        {"name": "gated decode", "op": "gated", "rows": 16, "n": 6400, "k": 4096, "groups": 1, "skew": 0.0,
         "act": "gelu", "save": False, "type": "bf16"},
        # gate/up of a training step over 8 experts, with what the backward pass needs
        {"name": "gated training", "op": "gated", "rows": 4096, "n": 14336, "k": 4096, "groups": 8, "skew": 0.5,
         "act": "silu", "save": True, "type": "bf16"},
        # the backward pass of that step
        {"name": "gated backward", "op": "gated_backward", "rows": 4096, "n": 14336, "k": 4096, "groups": 8,
         "skew": 0.5, "act": "silu", "type": "bf16"},
    ]


# the flops of the largest listed case, and the most weight elements a drawn case holds
MOST_FLOPS = 8 * 4096 * 14336 * 4096
MOST_WEIGHTS = 8 * 2 * 14336 * 4096


def draw(rng):
    def spread(lo, hi, step):
        return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step)

    while True:
        op = rng.choice(["quantize", "int8_product", "int8_gated", "product", "product_backward", "gated",
                         "gated_backward"])
        case = {"op": op, "rows": spread(1, 16384, 1), "k": spread(64, 14336, 16 if "int8" in op else 8),
                "type": rng.choice(["bf16", "fp16"])}
        if op != "quantize":
            case["n"] = spread(64, 14336, 8)
            case["groups"] = rng.choice([1, 1, 2, 5, 8, 16, 64])
            case["skew"] = rng.choice([0.0, 0.5, 1.0])
        if "gated" in op:
            case["act"] = rng.choice(["silu", "gelu"])
        if op == "gated":
            case["save"] = rng.random() < 0.5
        if op == "int8_product":
            case["type"] = rng.choice(["bf16", "fp16", "fp32"])
        cost = work(case)
        weights = case.get("groups", 0) * case.get("n", 0) * case["k"] * (2 if "gated" in op else 1)
        if cost["flops"] <= MOST_FLOPS and weights <= MOST_WEIGHTS:
            return case


def group_sizes(case):
    """Rows of each expert, the most popular first: shares (e + 1)^-skew, rounded by largest remainder."""
    share = [(e + 1.0) ** -case["skew"] for e in range(case["groups"])]
    ideal = [case["rows"] * s / sum(share) for s in share]
    sizes = [int(v) for v in ideal]
    order = sorted(range(len(ideal)), key=lambda e: (sizes[e] - ideal[e], e))
    for e in order[: case["rows"] - sum(sizes)]:
        sizes[e] += 1
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]
    rows, k, op = case["rows"], case["k"], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)

    def experts(n, std):
        # drawn expert by expert: the 32-bit draw is twice the size of what is kept
        return torch.stack([normal(n, k, std=std).to(dtype) for _ in range(case["groups"])])

    if op == "quantize":
        return {"case": case, "x": normal(rows, k).to(dtype)}

    # which expert is how popular differs from seed to seed; the sizes themselves are the case's
    sizes = group_sizes(case)
    order = torch.randperm(len(sizes), generator=torch.Generator().manual_seed(seed)).tolist()
    sizes = [sizes[i] for i in order]
    ends = [sum(sizes[: e + 1]) for e in range(len(sizes))]
    state = {"case": case, "ends": ends, "offsets": torch.tensor([0] + ends, dtype=torch.int32, device="cuda")}
    n = case["n"]
    wide = 2 * n if "gated" in op else n
    if op in ("int8_product", "int8_gated"):
        state["codes"], state["scale"] = quantize_plain(normal(rows, k))
        pairs = [quantize_plain(normal(wide, k, std=k ** -0.5)) for _ in range(case["groups"])]
        state["w"] = torch.stack([p[0] for p in pairs])
        state["w_scale"] = torch.stack([p[1] for p in pairs])
        return state
    state["x"] = normal(rows, k).to(dtype)
    state["w"] = experts(wide, k ** -0.5)
    if op == "product_backward":
        state["dy"] = normal(rows, n).to(dtype)
    if op == "gated_backward":
        state["dh"] = normal(rows, n).to(dtype)
        # what the forward pass of these inputs left
        state["gate_up"] = torch.empty(rows, wide, dtype=dtype, device="cuda")
        for e, (b, t) in enumerate(ranges(ends)):
            if t > b:
                state["gate_up"][b:t] = state["x"][b:t] @ state["w"][e].t()
    return state


def ranges(ends):
    return list(zip([0] + ends[:-1], ends))


def quantize_plain(x):
    # in 64 bits: the rounding chooses between two whole numbers
    wide = x.double()
    top = wide.abs().amax(dim=1, keepdim=True)
    codes = torch.round(wide * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return codes.to(torch.int8), (top[:, 0] / 127).float()


def act(name, g):
    if name == "silu":
        return g * (1 / (1 + torch.exp(-g)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def act_slope(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import expert_ffn_layer_router_amd as moe

    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        return moe.quantize_rows(s["x"])
    if op == "int8_product":
        return moe.int8_product(s["codes"], s["scale"], s["w"], s["w_scale"], s["offsets"], dtype=TYPES[case["type"]])
    if op == "int8_gated":
        return moe.int8_gated(s["codes"], s["scale"], s["w"], s["w_scale"], s["offsets"], activation=case["act"],
                              dtype=TYPES[case["type"]])
    if op == "product":
        return moe.expert_product(s["x"], s["w"], s["offsets"])
    if op == "product_backward":
        return moe.expert_product_backward(s["dy"], s["x"], s["w"], s["offsets"])
    if op == "gated":
        return moe.gated_product(s["x"], s["w"], s["offsets"], activation=case["act"], save=case["save"])
    return moe.gated_product_backward(s["dh"], s["gate_up"], s["x"], s["w"], s["offsets"], activation=case["act"])


def run_plain(s):
    case, op = s["case"], s["case"]["op"]
    dtype = TYPES[case["type"]]
    if op == "quantize":
        return quantize_plain(s["x"])
    n, rows = case["n"], case["rows"]
    dev = s["w"].device
    wide = s["w"].shape[1]
    if op in ("product_backward", "gated_backward"):
        if op == "gated_backward":
            g, u, dh = s["gate_up"][:, :n].float(), s["gate_up"][:, n:].float(), s["dh"].float()
            dy = torch.cat([dh * u * act_slope(case["act"], g), dh * act(case["act"], g)], dim=1)
        else:
            dy = s["dy"].float()
        dx = torch.empty_like(s["x"])
        dw = torch.zeros_like(s["w"])
        for e, (b, t) in enumerate(ranges(s["ends"])):
            if t > b:
                dx[b:t] = (dy[b:t] @ s["w"][e].float()).to(dtype)
                dw[e] = (dy[b:t].t() @ s["x"][b:t].float()).to(dtype)
        return dx, dw
    x = s["codes"] if "codes" in s else s["x"]
    y = torch.empty(rows, wide, dtype=torch.float32, device=dev)
    for e, (b, t) in enumerate(ranges(s["ends"])):
        if t > b:
            y[b:t] = x[b:t].float() @ s["w"][e].float().t()
            if "codes" in s:
                y[b:t] *= s["scale"][b:t, None] * s["w_scale"][e][None, :]
    if op in ("int8_product", "product"):
        return y.to(dtype)
    h = (act(case["act"], y[:, :n]) * y[:, n:]).to(dtype)
    return (h, y.to(dtype)) if case.get("save") else h


def work(case):
    rows, k, op = case["rows"], case["k"], case["op"]
    if op == "quantize":
        # read x; write the codes and one 32-bit scale a row; compare, scale and round each value
        return {"bytes": 2 * rows * k + rows * k + 4 * rows, "flops": 3 * rows * k}
    n, groups = case["n"], case["groups"]
    wide = 2 * n if "gated" in op else n
    used = sum(1 for c in group_sizes(case) if c)
    product = 2 * rows * wide * k
    offsets = 4 * (groups + 1)
    if op in ("int8_product", "int8_gated"):
        out = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
        return {"bytes": rows * k + 4 * rows + used * wide * (k + 4) + out * rows * n + offsets, "flops": product}
    if op in ("product", "gated"):
        kept = 2 * rows * wide if case.get("save") else 0
        return {"bytes": 2 * rows * k + 2 * used * wide * k + 2 * rows * n + kept + offsets, "flops": product}
    # backward: read dy (or dh and the saved pair), x and the used weights; write dx and every expert's dw
    read = 2 * rows * n + (2 * rows * wide if op == "gated_backward" else 0) + 2 * rows * k + 2 * used * wide * k
    return {"bytes": read + 2 * rows * k + 2 * groups * wide * k + offsets, "flops": 2 * product}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "quantize":
        codes, scales = [], []
        for part in s["x"].split(512):
            top = part.to(f64).abs().max(dim=1).values
            ratio = part.to(f64).mul(127).div(top.clamp_min(torch.finfo(f64).tiny)[:, None])
            low = torch.floor(ratio)
            rest = ratio - low  # a tie goes to the even neighbour
            up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2) == 1))
            codes.append((low + up.to(f64)).to(torch.int8))
            scales.append(top / 127)
        return torch.cat(codes), torch.cat(scales)
    n, rows, k = case["n"], case["rows"], case["k"]
    gated = "gated" in op
    parts, dws = [], []

    def curve(g):
        """act and its derivative."""
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            return g * sig, sig + g * sig * (1 - sig)
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * g + a * b * g * g * g)
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) * (a + 3 * a * b * g * g) / 2

    begin = 0
    for e, end in enumerate(s["ends"]):
        w = s["w"][e].to(f64)
        if op in ("product_backward", "gated_backward"):
            x = s["x"][begin:end].to(f64)
            if gated:
                g, u = s["gate_up"][begin:end].to(f64).split(n, dim=1)
                a, slope = curve(g)
                d = s["dh"][begin:end].to(f64)
                dy = torch.cat([d * u * slope, d * a], dim=1)
            else:
                dy = s["dy"][begin:end].to(f64)
            parts.append((torch.matmul(dy, w),))
            dws.append(torch.matmul(dy.t(), x) if end > begin else torch.zeros_like(w))
        else:
            x = (s["codes"] if "codes" in s else s["x"])[begin:end].to(f64)
            y = torch.matmul(x, w.t())
            if "codes" in s:
                y = y * s["scale"][begin:end].to(f64)[:, None] * s["w_scale"][e].to(f64)
            if gated:
                h = curve(y[:, :n])[0] * y[:, n:]
                parts.append((h, y) if case.get("save") else (h,))
            else:
                parts.append((y,))
        begin = end
    outs = tuple(torch.cat(p) for p in zip(*parts))
    if dws:
        return outs[0], torch.stack(dws)
    return outs if len(outs) > 1 else outs[0]
