"""Products of experts in 8-bit floating point, and the step that trains them, as cases to measure.

Codes are e4m3 with one 32-bit scale for each block of 128: rows (activations, gradients) have a scale for every 128
consecutive values of a row, scale[b, r]; weights one for every 128 x 128 values, w_scale[e, i, b].  Rows that belong to
one expert stand together (the order that the layer's regroup leaves): group e owns rows offsets[e] .. offsets[e + 1] - 1.

  quantize          scale = a / 448, codes = x 448 / a rounded to e4m3, a the block's largest magnitude
  product           y[r, n] = sum_b scale[b, r] w_scale[e, n // 128, b] sum_{k in b} codes[r, k] w[e, n, k]
  gated             h = act(g) u, g and u the products with w[e, 0] and w[e, 1]; (g, u) too where a step trains
  product_backward  dx = dy w[e], dy in codes with a scale for every 128 of its n columns
  gated_backward    dg = dh u act'(g), du = dh act(g), both returned and put into codes; dx = dg w[e, 0] + du w[e, 1]
  adamw             m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
                    p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
                    for many tensors; m and v in 32 bits, or in 8 (m e4m3, v e5m2) with a scale for every 128 values
                    and rounded up or down at random, by numbers that follow from the seed, the step, the tensor's and
                    the value's number

With `own` false, `run` computes them in elementary torch operations in 32 bits (the codes, whose rounding decides
between two neighbours, in 64); with `own` true it calls the framework's kernels.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
STEP, SEED = 10, 20260101
HYPER = {"lr": 1e-4, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.01}


def listed():
    return [
        # one decode step's hidden states (16 tokens), put into codes for the experts' products
        {"name": "quantize decode", "op": "quantize", "tiles": False, "groups": 1, "rows": 16, "k": 4096,
         "type": "bf16"},
        # the gate and up weights of 8 experts, put into codes after a training step or when they are loaded
        {"name": "quantize weights", "op": "quantize", "tiles": True, "groups": 16, "rows": 14336, "k": 4096,
         "type": "bf16"},
        # one token through one fine-grained expert's down projection: the smallest call, latency counts
        {"name": "product one row", "op": "product", "rows": 1, "n": 4096, "k": 2048, "groups": 1, "skew": 0.0,
         "type": "bf16"},
        # the down projection of a 2048-token, top-2 prefill chunk over 8 experts
        {"name": "product prefill", "op": "product", "rows": 4096, "n": 4096, "k": 14336, "groups": 8, "skew": 0.5,
         "type": "bf16"},
        # gate/up of a 16-token, top-2 decode step over 8 experts: bound by the weights' bytes
        {"name": "gated decode", "op": "gated", "rows": 32, "n": 14336, "k": 4096, "groups": 8, "skew": 0.5,
         "act": "silu", "save": False, "type": "bf16"},
        # gate/up of a training step over 8 experts, with what the backward pass needs
        {"name": "gated training", "op": "gated", "rows": 4096, "n": 14336, "k": 4096, "groups": 8, "skew": 0.5,
         "act": "silu", "save": True, "type": "bf16"},
        # a short batch through a narrow block of odd widths, whose last blocks of 128 are partial
        {"name": "product backward odd", "op": "product_backward", "rows": 77, "n": 1008, "k": 1424, "groups": 3,
         "skew": 0.8, "type": "fp16"},
        # the rows' gradient where 64 fine-grained experts train: short ragged groups
        {"name": "product backward fine", "op": "product_backward", "rows": 24576, "n": 4096, "k": 2048, "groups": 64,
         "skew": 1.0, "type": "bf16"},
        # the gated block's backward pass in a small batch of odd widths
        {"name": "gated backward odd", "op": "gated_backward", "rows": 300, "n": 1008, "k": 1424, "groups": 5,
         "skew": 1.0, "act": "gelu", "type": "fp16"},
        # and that of the training step above
        {"name": "gated backward", "op": "gated_backward", "rows": 4096, "n": 14336, "k": 4096, "groups": 8,
         "skew": 0.5, "act": "silu", "type": "bf16"},
        # the weights of two small layers of odd sizes, everything in 32 bits: the smallest step
        {"name": "adamw small", "op": "adamw", "layers": 2, "experts": 3, "d": 63, "f": 131, "type": "fp32",
         "grad": "fp32", "bits": 32, "master": False},
        # the weights of one layer of 8 experts in 16 bits, with a copy in 32 and states in 8
        {"name": "adamw experts", "op": "adamw", "layers": 1, "experts": 8, "d": 4096, "f": 6400, "type": "bf16",
         "grad": "bf16", "bits": 8, "master": True},
    ]


# the most flops of a listed product, weights of a drawn one, and values of a listed step
MOST_FLOPS = 2 * 4096 * 2 * 14336 * 4096
MOST_WEIGHTS = 8 * 2 * 14336 * 4096
MOST_VALUES = 3 * 8 * 4096 * 6400


def draw(rng):
    def spread(lo, hi, step):
        return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step)

    while True:
        op = rng.choice(["quantize", "product", "gated", "product_backward", "gated_backward", "adamw"])
        if op == "adamw":
            kind = rng.choice(["bf16", "fp16", "fp32"])
            case = {"op": op, "layers": rng.choice([1, 2]), "experts": rng.choice([1, 3, 8, 16]),
                    "d": spread(16, 4096, 1), "f": spread(16, 14336, 1), "type": kind,
                    "grad": rng.choice([kind, "fp32"]), "bits": rng.choice([8, 32]),
                    "master": kind != "fp32" and rng.random() < 0.5}
            if sum(math.prod(s) for s in tensor_shapes(case)) <= MOST_VALUES:
                return case
            continue
        case = {"op": op, "rows": spread(1, 16384, 1), "k": spread(64, 14336, 16),
                "groups": rng.choice([1, 1, 2, 5, 8, 16, 64]), "type": rng.choice(["bf16", "fp16"])}
        if op == "quantize":
            case["tiles"] = rng.random() < 0.5
            case["groups"] = case["groups"] if case["tiles"] else 1
            if case["groups"] * case["rows"] * case["k"] <= MOST_WEIGHTS:
                return case
            continue
        case["n"] = spread(64, 14336, 16)
        case["skew"] = rng.choice([0.0, 0.5, 1.0])
        if "gated" in op:
            case["act"] = rng.choice(["silu", "gelu"])
        if op == "gated":
            case["save"] = rng.random() < 0.5
        weights = case["groups"] * case["n"] * case["k"] * (2 if "gated" in op else 1)
        if work(case)["flops"] <= MOST_FLOPS and weights <= MOST_WEIGHTS:
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


def tensor_shapes(case):
    """The weights of a step: of each layer the router, its bias, and the experts' two matrices."""
    e, d, f = case["experts"], case["d"], case["f"]
    return [(e, d), (e,), (e, 2 * f, d), (e, d, f)] * case["layers"]


def blocks(n):
    return (n + 127) // 128


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]
    op = case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)

    if op == "adamw":
        state = {"case": case, "m": [], "v": [], "m_scale": [], "v_scale": [], "params": [], "grads": [], "master": []}
        for shape in tensor_shapes(case):
            std = shape[-1] ** -0.5
            wide = normal(*shape, std=std)
            state["params"].append(wide.to(dtype))
            if case["master"]:
                state["master"].append(wide)
            # sizes of gradients differ from row to row by a factor of some ten, as tokens and experts do
            spread = torch.exp(normal(*shape[:-1], 1))
            state["grads"].append((normal(*shape, std=1e-3) * spread).to(TYPES[case["grad"]]))
            m, v = normal(*shape, std=3e-4) * spread, (normal(*shape, std=1e-3) * spread).square_()
            if case["bits"] == 8:
                m, m_scale = states_into_codes(m, E4M3, None)
                v, v_scale = states_into_codes(v, E5M2, None)
                state["m_scale"].append(m_scale)
                state["v_scale"].append(v_scale)
            state["m"].append(m)
            state["v"].append(v)
        return state

    rows, k = case["rows"], case["k"]
    if op == "quantize":
        x = torch.stack([normal(rows, k).to(dtype) for _ in range(case["groups"])])
        return {"case": case, "x": x if case["tiles"] else x[0]}

    # which expert is how popular differs from seed to seed; the sizes themselves are the case's
    sizes = group_sizes(case)
    order = torch.randperm(len(sizes), generator=torch.Generator().manual_seed(seed)).tolist()
    sizes = [sizes[i] for i in order]
    ends = [sum(sizes[: e + 1]) for e in range(len(sizes))]
    state = {"case": case, "ends": ends, "offsets": torch.tensor([0] + ends, dtype=torch.int32, device="cuda")}
    n = case["n"]
    halves = (2,) if "gated" in op else ()
    # drawn expert by expert: the draw in 32 bits is four times the size of what is kept
    experts = [tiles_into_codes(normal(*halves, n, k, std=k ** -0.5)) for _ in range(case["groups"])]
    state["w"] = torch.stack([c.view(torch.uint8) for c, _ in experts]).view(E4M3)
    state["w_scale"] = torch.stack([s for _, s in experts])
    if op == "product_backward":
        state["codes"], state["scale"] = rows_into_codes(normal(rows, n))
    elif op == "gated_backward":
        state["dh"] = normal(rows, n).to(dtype)
        state["gate_up"] = normal(rows, 2 * n).to(dtype)
    else:
        state["codes"], state["scale"] = rows_into_codes(normal(rows, k))
    return state


def ranges(ends):
    return list(zip([0] + ends[:-1], ends))


def padded(x, *sizes):
    """x with zeros behind its last dimensions, up to whole blocks."""
    out = x.new_zeros(x.shape[: x.dim() - len(sizes)] + sizes)
    out[(...,) + tuple(slice(0, s) for s in x.shape[x.dim() - len(sizes):])] = x
    return out


def into_codes(x, top):
    """x 448 / top as e4m3, in 64 bits before the rounding, and top / 448."""
    x = x.double() * (448 / torch.where(top > 0, top, torch.ones_like(top)).double())
    return x.float().to(E4M3), top / 448


def rows_into_codes(x):
    rows, k = x.shape
    whole = padded(x.float(), blocks(k) * 128).view(rows, blocks(k), 128)
    codes, scale = into_codes(whole, whole.abs().amax(dim=2, keepdim=True))
    return codes.view(rows, -1)[:, :k].contiguous(), scale.view(rows, -1).t().contiguous()


def tiles_into_codes(x):
    n, k = x.shape[-2:]
    whole = padded(x.float(), blocks(n) * 128, blocks(k) * 128).view(*x.shape[:-2], blocks(n), 128, blocks(k), 128)
    codes, scale = into_codes(whole, whole.abs().amax(dim=(-3, -1), keepdim=True))
    codes = codes.view(*x.shape[:-2], blocks(n) * 128, blocks(k) * 128)[..., :n, :k]
    return codes.contiguous(), scale.squeeze(-1).squeeze(-2)


def rows_of(codes, scale):
    """The values of rows of codes."""
    return codes.float() * scale.t().repeat_interleave(128, dim=1)[:, : codes.shape[1]]


def tiles_of(codes, scale):
    """The values of weights in codes."""
    n, k = codes.shape[-2:]
    return codes.float() * scale.repeat_interleave(128, dim=-2)[..., :n, :].repeat_interleave(128, dim=-1)[..., :k]


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


# the random numbers of an 8-bit step: 32 bits for each value, from two multiplications whose halves are folded
LOW = 0xFFFFFFFF


def fold(x, by):
    p = x * by  # the low 64 bits
    return ((p >> 32) ^ p) & LOW


def mixed(x, key):
    return fold((fold(x ^ key, 0x9E3779B9) + key) & LOW, 0xBB67AE85)


def random_of(numel, tensor, device):
    key = SEED & LOW
    for part in (SEED >> 32, STEP, tensor, 0):  # 0: the high half of the values' numbers, which are below 2^32 here
        key = int(mixed(torch.tensor(part), key))
    return mixed(torch.arange(numel, device=device), key)


def power_of_two(e):
    return ((e + 127) << 23).view(torch.float32)


def states_into_codes(x, kind, random):
    """Codes of a state and their scales, of each 128 consecutive values; random: 16 bits for each value, that round
    its code up or down, or None: to the nearest.  Squares' codes (e5m2) of values above zero are not zero."""
    most, lowest, bits = (448.0, -6, 3) if kind is E4M3 else (57344.0, -14, 2)
    flat = x.reshape(-1)
    whole = padded(flat, blocks(flat.numel()) * 128).view(-1, 128)
    scale = whole.abs().amax(dim=1, keepdim=True) / most
    y = whole / torch.where(scale > 0, scale, torch.ones_like(scale))
    # a code's unit in its last place
    unit = torch.frexp(y)[1].sub_(1).clamp_(min=lowest).sub_(bits)
    y = y * power_of_two(-unit)
    n = y.abs()
    if random is None:
        n = torch.round(n)
    else:
        n = torch.floor(n + padded(random, whole.numel()).view(-1, 128).float() / 65536)
    if kind is E5M2:
        n = torch.where((n == 0) & (whole > 0), torch.ones_like(n), n)
    codes = (n * power_of_two(unit)).clamp_(max=most).copysign_(y).to(kind)
    return codes.view(-1)[: flat.numel()].view(x.shape), scale.view(-1)


def states_of(codes, scale):
    whole = padded(codes.reshape(-1).float(), scale.numel() * 128).view(-1, 128) * scale[:, None]
    return whole.view(-1)[: codes.numel()].view(codes.shape)


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import expert_ffn_layer_router_amd as moe

    case, op = s["case"], s["case"]["op"]
    if op == "adamw":
        eight = {"m_scale": s["m_scale"], "v_scale": s["v_scale"], "seed": SEED} if case["bits"] == 8 else {}
        moe.adamw_step(s["params"], s["grads"], s["m"], s["v"], STEP, master=s["master"] or None, **eight, **HYPER)
        return {k: s[k] for k in ("params", "master", "m", "v", "m_scale", "v_scale")}
    if op == "quantize":
        return moe.quantize_blocks(s["x"], tiles=case["tiles"])
    if op == "product":
        return moe.fp8_product(s["codes"], s["scale"], s["w"], s["w_scale"], s["offsets"], dtype=TYPES[case["type"]])
    if op == "gated":
        return moe.fp8_gated(s["codes"], s["scale"], s["w"], s["w_scale"], s["offsets"], activation=case["act"],
                             save=case["save"], dtype=TYPES[case["type"]])
    if op == "product_backward":
        return moe.fp8_product_backward(s["codes"], s["scale"], s["w"], s["w_scale"], s["offsets"],
                                        dtype=TYPES[case["type"]])
    return moe.fp8_gated_backward(s["dh"], s["gate_up"], s["w"], s["w_scale"], s["offsets"], activation=case["act"])


def run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "adamw":
        return adamw_plain(s)
    if op == "quantize":
        return tiles_into_codes(s["x"]) if case["tiles"] else rows_into_codes(s["x"])
    dtype, n, rows = TYPES[case["type"]], case["n"], case["rows"]
    slopes = None
    if op == "gated_backward":
        g, u, dh = s["gate_up"][:, :n].float(), s["gate_up"][:, n:].float(), s["dh"].float()
        halves = [dh * u * act_slope(case["act"], g), dh * act(case["act"], g)]
        slopes = torch.cat(halves, dim=1).to(dtype)
        x = torch.cat([rows_of(*rows_into_codes(half)) for half in halves], dim=1)
    else:
        x = rows_of(s["codes"], s["scale"])
    wide = case["k"] if "backward" in op else 2 * n if op == "gated" else n
    y = torch.empty(rows, wide, dtype=torch.float32, device=x.device)
    for e, (b, t) in enumerate(ranges(s["ends"])):
        if t > b:
            w = tiles_of(s["w"][e], s["w_scale"][e]).view(-1, case["k"])
            torch.mm(x[b:t], w if "backward" in op else w.t(), out=y[b:t])
    if op == "gated_backward":
        return y.to(dtype), slopes
    if op == "gated":
        h = (act(case["act"], y[:, :n]) * y[:, n:]).to(dtype)
        return (h, y.to(dtype)) if case["save"] else h
    return y.to(dtype)


def adamw_plain(s):
    case = s["case"]
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    for i, p in enumerate(s["params"]):
        g = s["grads"][i].float()
        eight = case["bits"] == 8
        m = states_of(s["m"][i], s["m_scale"][i]) if eight else s["m"][i]
        v = states_of(s["v"][i], s["v_scale"][i]) if eight else s["v"][i]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + (g * g) * (1 - b2)
        wide = s["master"][i] if case["master"] else p.float()
        new = wide * (1 - lr * HYPER["weight_decay"])
        new -= (lr / (1 - b1 ** STEP)) * m / (torch.sqrt(v) / math.sqrt(1 - b2 ** STEP) + HYPER["eps"])
        p.copy_(new)
        if case["master"]:
            s["master"][i].copy_(new)
        if eight:
            random = random_of(p.numel(), i, p.device)
            m, m_scale = states_into_codes(m, E4M3, random & 0xFFFF)
            v, v_scale = states_into_codes(v, E5M2, random >> 16)
            s["m_scale"][i].copy_(m_scale)
            s["v_scale"][i].copy_(v_scale)
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
    return {k: s[k] for k in ("params", "master", "m", "v", "m_scale", "v_scale")}


SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    op = case["op"]
    if op == "adamw":
        values = sum(math.prod(s) for s in tensor_shapes(case))
        size = SIZES[case["type"]]
        # the weights in and out (with a copy in 32 bits: that in and out, the weights out), the gradients in
        each = (8 + size if case["master"] else 2 * size) + SIZES[case["grad"]]
        # both states in and out
        each += 16 if case["bits"] == 32 else 4 * (1 + 4 / 128)
        return {"bytes": each * values, "flops": 15 * values}
    rows, k = case["rows"], case["k"]
    if op == "quantize":
        values = case["groups"] * rows * k
        return {"bytes": 3 * values + 4 * values / (128 * 128 if case["tiles"] else 128), "flops": 3 * values}
    n, groups = case["n"], case["groups"]
    wide = 2 * n if "gated" in op else n
    used = sum(1 for c in group_sizes(case) if c)
    weights = used * (wide * k + 4 * (wide // n) * blocks(n) * blocks(k)) + 4 * (groups + 1)
    size = SIZES[case["type"]]
    if op in ("product", "gated"):
        ends = rows * (k + 4 * blocks(k)) + size * rows * n + (size * rows * wide if case.get("save") else 0)
    elif op == "product_backward":
        ends = rows * (n + 4 * blocks(n)) + size * rows * k
    else:  # dh and (g, u) in, (dg, du) and dx out
        ends = size * rows * (n + 2 * wide + k)
    return {"bytes": weights + ends, "flops": 2 * rows * wide * k}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]

    def grid(q, lowest, bits):
        """The step of an 8-bit float's codes around q."""
        e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -60))).clamp_min(lowest)
        return torch.exp2(e - bits)

    def rows64(x, top_only=False):
        """Codes and scales of rows, block by block."""
        codes, scales = torch.empty_like(x), []
        for at in range(0, x.shape[1], 128):
            part = x[:, at:at + 128]
            top = part.abs().max(dim=1).values
            scales.append(top / 448)
            q = part * 448 / top.clamp_min(torch.finfo(f64).tiny)[:, None]
            step = grid(q, -6, 3)
            codes[:, at:at + 128] = torch.round(q / step) * step
        return codes, torch.stack(scales)

    if op == "quantize":
        if not case["tiles"]:
            return rows64(s["x"].to(f64))
        n, k = case["rows"], case["k"]
        codes = torch.empty(s["x"].shape, dtype=torch.float32, device="cuda")  # e4m3 values fit exactly
        scales = torch.empty(case["groups"], blocks(n), blocks(k), dtype=f64, device="cuda")
        for e in range(case["groups"]):
            for i in range(blocks(n)):
                part = s["x"][e, 128 * i:128 * i + 128].to(f64)
                tops = torch.stack([c.abs().max() for c in part.split(128, dim=1)])
                scales[e, i] = tops / 448
                q = part * 448 / tops.clamp_min(torch.finfo(f64).tiny).repeat_interleave(128)[:k]
                step = grid(q, -6, 3)
                codes[e, 128 * i:128 * i + 128] = (torch.round(q / step) * step).float()
        return codes, scales

    if op == "adamw":
        out = {key: [] for key in ("params", "master", "m", "v", "m_scale", "v_scale")}
        (b1, b2), lr = HYPER["betas"], HYPER["lr"]

        def state64(codes, scale):
            if scale is None:
                return codes.to(f64)
            flat = codes.to(torch.float32).to(f64).reshape(-1)
            return (flat * scale.to(f64).repeat_interleave(128)[: flat.numel()]).view(codes.shape)

        def coded(x, most, lowest, bits, u):
            flat = x.reshape(-1)
            count = -(-flat.numel() // 128)
            room = flat.new_zeros(count * 128)
            room[: flat.numel()] = flat
            scale = room.view(count, 128).abs().max(dim=1).values / most
            q = flat.abs() / scale.clamp_min(torch.finfo(f64).tiny).repeat_interleave(128)[: flat.numel()]
            step = grid(q, lowest, bits)
            n = torch.floor(q / step + u)
            if bits == 2:
                n = torch.where((n < 1) & (flat > 0), torch.ones_like(n), n)
            return ((n * step).clamp_max(most) * torch.sign(flat)).float().view(x.shape), scale

        for i in range(len(s["params"])):
            scales = (s["m_scale"][i], s["v_scale"][i]) if case["bits"] == 8 else (None, None)
            g = s["grads"][i].to(f64)
            m = b1 * state64(s["m"][i], scales[0]) + (1 - b1) * g
            v = b2 * state64(s["v"][i], scales[1]) + (1 - b2) * g.square()
            p = (s["master"] or s["params"])[i].to(f64)
            rate = (m / (1 - b1 ** STEP)) / ((v / (1 - b2 ** STEP)).sqrt() + HYPER["eps"])
            p = p - lr * HYPER["weight_decay"] * p - lr * rate
            out["params"].append(p)
            if case["master"]:
                out["master"].append(p)
            if case["bits"] == 8:
                draws = random_of(p.numel(), i, p.device)
                for key, x, args, u in (("m", m, (448.0, -6, 3), draws % 65536),
                                        ("v", v, (57344.0, -14, 2), draws // 65536)):
                    codes, scale = coded(x, *args, u.to(f64) / 65536)
                    out[key].append(codes)
                    out[key + "_scale"].append(scale)
            else:
                out["m"].append(m)
                out["v"].append(v)
        return out

    n, rows, k = case["n"], case["rows"], case["k"]

    def curve(g):
        """act and its derivative."""
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            return g * sig, sig + g * sig * (1 - sig)
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * g + a * b * g * g * g)
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) * (a + 3 * a * b * g * g) / 2

    def row_values(codes, scale):
        x = codes.to(f64)
        for b in range(scale.shape[0]):
            x[:, 128 * b:128 * b + 128] *= scale[b].to(f64)[:, None]
        return x

    def weight_values(codes, scale):
        x = codes.to(torch.float32).to(f64)
        for i in range(scale.shape[0]):
            x[128 * i:128 * i + 128] *= scale[i].to(f64).repeat_interleave(128)[: x.shape[1]]
        return x

    slopes = None
    if op == "gated_backward":
        g, u = s["gate_up"].to(f64).split(n, dim=1)
        a, slope = curve(g)
        d = s["dh"].to(f64)
        slopes = (d * u * slope, d * a)
        x = [row_values(*rows64(half)) for half in slopes]
    else:
        x = [row_values(s["codes"].to(torch.float32), s["scale"])]
    parts, begin = [], 0
    for e, end in enumerate(s["ends"]):
        if "gated" in op:
            w = [weight_values(s["w"][e][i], s["w_scale"][e][i]) for i in (0, 1)]
        else:
            w = [weight_values(s["w"][e], s["w_scale"][e])]
        if "backward" in op:
            y = sum(torch.matmul(xi[begin:end], wi) for xi, wi in zip(x, w))
            parts.append((y,))
        elif op == "gated":
            g, u = (torch.matmul(x[0][begin:end], wi.t()) for wi in w)
            parts.append((curve(g)[0] * u, torch.cat([g, u], dim=1))[: 2 if case["save"] else 1])
        else:
            parts.append((torch.matmul(x[0][begin:end], w[0].t()),))
        begin = end
    outs = tuple(torch.cat(p) for p in zip(*parts))
    if slopes is not None:
        return outs[0], torch.cat(slopes, dim=1)
    return outs if len(outs) > 1 else outs[0]
