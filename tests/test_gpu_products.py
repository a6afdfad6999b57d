"""The grouped products on the GPU against plain 64-bit ones.

Bounds, per element, from the roundings alone (u = half a step of the output's
type relative to the value, 2^-8 bf16, 2^-11 fp16, 2^-24 fp32; e = 2^-24):
  sums     16-bit operands: products are exact in fp32; K additions, in any
           order and blocking, each off by at most one step (2e: a matrix core
           may truncate) of a partial sum no larger than S = sum |x w|:
           2 K e S
  codes    the int32 sum is exact; its conversion and two scalings: 3e |y|
  act(g)   exp2 and reciprocal within 2 steps each, z log2(e) within one
           (times |z| in the exponential), and a few fp32 operations:
           A = 2e (8 + 4 |z|) |act(g)|, z the sigmoid's argument;
           the error d of g itself moves act(g) by at most 1.13 d
  output   u |value|, and half of the smallest subnormal in fp16 (2^-25)
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


def half_step(torch, dtype):
    return torch.finfo(dtype).eps / 2


def rounded(torch, value, before, dtype):
    """Bound of the output: the error before rounding, plus the rounding."""
    return before + half_step(torch, dtype) * (value.abs() + before) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check(torch, got, ref, bound, what):
    assert got.shape == ref.shape, what
    off = (got.double() - ref).abs()
    worst = (off - bound).max().item() if off.numel() else -1.0
    if not worst <= 0:  # NaN fails too
        i = (off - bound).nan_to_num(nan=float("inf")).argmax().item()
        raise AssertionError(f"{what}: element {np.unravel_index(i, tuple(got.shape))}: got {got.flatten()[i].item()!r} "
                             f"expected {ref.flatten()[i].item()!r} within {bound.flatten()[i].item():.3g}")


class Case:
    """Inputs of one grouped product; sizes are rows per group, `before` and
    `after` rows that belong to none."""

    def __init__(self, torch, sizes, n, k, dtype, wide=1, before=0, after=0, seed=0, offsets=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.sizes, self.n, self.k, self.dtype = torch, sizes, n, k, dtype
        self.rows = before + sum(sizes) + after
        ends = [before]
        for s in sizes:
            ends.append(ends[-1] + s)
        self.ends = ends
        self.offsets = torch.tensor(ends, dtype=torch.int32, device="cuda") if offsets else None
        self.wide = wide * n
        self.gen = gen
        self.x = self.normal(self.rows, k)
        self.w = self.normal(len(sizes), self.wide, k, std=k ** -0.5)

    def normal(self, *shape, std=1.0):
        torch = self.torch
        return (torch.randn(*shape, generator=self.gen, device="cuda") * std).to(self.dtype)

    def groups(self):
        return [(e, self.ends[e], self.ends[e + 1]) for e in range(len(self.sizes)) if self.sizes[e]]

    def forward(self):
        """(y, bound of its sums) in 64 bits; rows of no group are zero."""
        torch = self.torch
        y = torch.zeros(self.rows, self.wide, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(y)
        for e, b, t in self.groups():
            x, w = self.x[b:t].double(), self.w[e].double().t().contiguous()
            y[b:t] = x @ w
            s[b:t] = x.abs() @ w.abs()
        return y, 2 * self.k * E * s

    def member(self):
        m = self.torch.zeros(self.rows, dtype=self.torch.bool, device="cuda")
        m[self.ends[0]:self.ends[-1]] = True
        return m


def act64(torch, name, g):
    """(value, slope, |z|, |g z' s (1 - s)|) in 64 bits."""
    c, b = 1.5957691216057308, 0.044715
    z, dz = (g, torch.ones_like(g)) if name == "silu" else (c * (g + b * g ** 3), c * (1 + 3 * b * g * g))
    s = torch.sigmoid(z)
    curve = g * s * torch.sigmoid(-z) * dz
    return g * s, s + curve, z.abs(), curve.abs()


def gated64(torch, act, g, u, dg, du):
    """h and the bound before its rounding, for g and u within dg and du."""
    a, _, z, _ = act64(torch, act, g)
    da = 1.13 * dg + 2 * E * (8 + 4 * z) * a.abs()
    h = a * u
    return h, da * u.abs() + (a.abs() + da) * du + 2 * E * h.abs()


TYPES = ["bfloat16", "float16"]

# sizes, n, k: one row to several tiles, empty groups, partial tiles, widths
# that end inside a 32-column, 128-column and 64-byte step
FEW = [([1], 8, 8), ([1], 64, 4096), ([3], 1000, 72), ([16], 40, 136), ([17], 24, 64), ([33], 264, 2056),
       ([64], 128, 520), ([0, 1, 0, 5, 16, 0, 7], 72, 200), ([20, 0, 44], 136, 328)]
TILES = [([65], 8, 8), ([129], 136, 72), ([200], 1000, 1416), ([0, 70, 0, 1, 128, 255, 0], 264, 200),
         ([256, 300], 128, 64), ([1000], 392, 456), ([3, 130, 67], 1000, 2056)]
# many groups with more rows than the streaming kernel takes: tiles at small widths; and uneven
# groups of few rows on average, whose blocks walk over a group's row tiles
MANY = [([150] + [0] * 8, 8, 16), ([0, 70, 0, 1, 128, 255, 0, 0, 0, 0], 264, 200), ([1000] + [0] * 8, 392, 464),
        ([0] * 8 + [200], 1000, 1416), ([3, 130, 67] + [0] * 7, 1000, 2056), ([0, 300] + [0] * 8, 264, 8200),
        ([0] * 20 + [700] + [3] * 30 + [0] * 13, 264, 80), ([1, 150] + [7] * 14, 1032, 520)]
# past the streaming kernel: 128-wide blocks (whole, and with the contraction split), 256-wide ones (the
# remainder of the last round split in the last)
BIG = [([3700], 4096, 72), ([500, 0, 1, 1255, 129, 1100], 1000, 2056), ([2049], 520, 4104), ([4096], 4096, 72),
       ([511, 0, 1300, 257, 700, 130], 2568, 136), ([3000, 1, 900], 4104, 4104)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + MANY + BIG, ids=str)
def test_expert_product(torch, moe, sizes, n, k, dtype):
    say(f"expert_product {sizes} {n} {k} {dtype}")
    c = Case(torch, sizes, n, k, getattr(torch, dtype))
    y, before = c.forward()
    got = moe.expert_product(c.x, c.w, c.offsets)
    check(torch, got, y, rounded(torch, y, before, c.dtype), "y")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + MANY + BIG[1:], ids=str)
def test_gated_product(torch, moe, sizes, n, k, dtype, act):
    say(f"gated_product {sizes} {n} {k} {dtype} {act}")
    c = Case(torch, sizes, n, k, getattr(torch, dtype), wide=2)
    y, before = c.forward()
    h, h_before = gated64(torch, act, y[:, :n], y[:, n:], before[:, :n], before[:, n:])
    got, gu = moe.gated_product(c.x, c.w, c.offsets, activation=act, save=True)
    check(torch, got, h, rounded(torch, h, h_before, c.dtype), "h")
    check(torch, gu, y, rounded(torch, y, before, c.dtype), "gate_up")
    alone = moe.gated_product(c.x, c.w, c.offsets, activation=act)
    assert torch.equal(alone, got)


def grads64(torch, c, dy, dy_off):
    """dx, dw and the bounds before their rounding, for dy within dy_off."""
    dx = torch.zeros(c.rows, c.k, dtype=torch.float64, device="cuda")
    dw = torch.zeros(len(c.sizes), c.wide, c.k, dtype=torch.float64, device="cuda")
    dx_off, dw_off = torch.zeros_like(dx), torch.zeros_like(dw)
    for e, b, t in c.groups():
        x, w, d, o = c.x[b:t].double(), c.w[e].double(), dy[b:t], dy_off[b:t]
        dt, ot = d.t().contiguous(), o.t().contiguous()
        dx[b:t] = d @ w
        dx_off[b:t] = (o + 2 * c.wide * E * (d.abs() + o)) @ w.abs()
        dw[e] = dt @ x
        dw_off[e] = (ot + 2 * (t - b) * E * (dt.abs() + ot)) @ x.abs()
    return dx, dw, dx_off, dw_off


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + BIG, ids=str)
def test_expert_product_backward(torch, moe, sizes, n, k, dtype):
    say(f"expert_product_backward {sizes} {n} {k} {dtype}")
    c = Case(torch, sizes, n, k, getattr(torch, dtype))
    dy = c.normal(c.rows, n)
    dx, dw, dx_off, dw_off = grads64(torch, c, dy.double(), torch.zeros(c.rows, n, dtype=torch.float64, device="cuda"))
    got_dx, got_dw = moe.expert_product_backward(dy, c.x, c.w, c.offsets)
    check(torch, got_dx, dx, rounded(torch, dx, dx_off, c.dtype), "dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, c.dtype), "dw")
    none, wide = moe.expert_product_backward(dy, c.x, c.w, c.offsets, need_dx=False, dw_dtype=torch.float32)
    assert none is None and wide.dtype == torch.float32
    check(torch, wide, dw, rounded(torch, dw, dw_off, torch.float32), "dw fp32")
    again, none = moe.expert_product_backward(dy, c.x, c.w, c.offsets, need_dw=False)
    assert none is None and torch.equal(again, got_dx)


def slopes64(torch, act, dh, gu, n, dtype):
    """(dg, du) from the saved (g, u), and how far the kernel's rounded ones may be."""
    g, u, d = gu[:, :n].double(), gu[:, n:].double(), dh.double()
    a, slope, z, curve = act64(torch, act, g)
    s = slope - curve * torch.sign(g)  # the sigmoid
    dg, du = d * u * slope, d * a
    dg_off = (d * u).abs() * 2 * E * (16 + 8 * z) * (s.abs() + curve) + 4 * E * dg.abs()
    du_off = d.abs() * 2 * E * (8 + 4 * z) * a.abs() + 2 * E * du.abs()
    dy, off = torch.cat([dg, du], 1), torch.cat([dg_off, du_off], 1)
    return dy, rounded(torch, dy, off, dtype)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + BIG[1:], ids=str)
def test_gated_product_backward(torch, moe, sizes, n, k, dtype, act):
    say(f"gated_product_backward {sizes} {n} {k} {dtype} {act}")
    c = Case(torch, sizes, n, k, getattr(torch, dtype), wide=2)
    dh = c.normal(c.rows, n)
    gu = c.normal(c.rows, 2 * n, std=2.0)
    dy, off = slopes64(torch, act, dh, gu, n, c.dtype)
    dx, dw, dx_off, dw_off = grads64(torch, c, dy, off)
    got_dx, got_dw = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, activation=act)
    check(torch, got_dx, dx, rounded(torch, dx, dx_off, c.dtype), "dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, c.dtype), "dw")


def int_case(torch, sizes, n, k, wide, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = Case(torch, sizes, n, 16, torch.bfloat16, wide=wide)
    c.k = k
    c.x = torch.randint(-128, 128, (c.rows, k), generator=gen, device="cuda").to(torch.int8)
    c.w = torch.randint(-128, 128, (len(sizes), c.wide, k), generator=gen, device="cuda").to(torch.int8)
    c.scale = torch.rand(c.rows, generator=gen, device="cuda") * 0.02
    c.w_scale = torch.rand(len(sizes), c.wide, generator=gen, device="cuda") * (0.02 * k ** -0.5)
    y = torch.zeros(c.rows, c.wide, dtype=torch.float64, device="cuda")
    for e, b, t in c.groups():
        y[b:t] = (c.x[b:t].double() @ c.w[e].double().t().contiguous()) * c.scale[b:t].double()[:, None] * c.w_scale[e].double()
    return c, y


def to16(cases):
    return [(s, n, max(16, k // 16 * 16)) for s, n, k in cases]


@pytest.mark.parametrize("dtype", TYPES + ["float32"])
@pytest.mark.parametrize("sizes,n,k", to16(FEW + TILES + MANY + BIG), ids=str)
def test_int8_product(torch, moe, sizes, n, k, dtype):
    say(f"int8_product {sizes} {n} {k} {dtype}")
    c, y = int_case(torch, sizes, n, k, 1)
    t = getattr(torch, dtype)
    got = moe.int8_product(c.x, c.scale, c.w, c.w_scale, c.offsets, dtype=t)
    check(torch, got, y, rounded(torch, y, 3 * E * y.abs(), t), "y")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", to16(FEW + TILES + MANY + [BIG[1]]), ids=str)
def test_int8_gated(torch, moe, sizes, n, k, dtype, act):
    say(f"int8_gated {sizes} {n} {k} {dtype} {act}")
    c, y = int_case(torch, sizes, n, k, 2)
    t = getattr(torch, dtype)
    off = 3 * E * y.abs()
    h, before = gated64(torch, act, y[:, :n], y[:, n:], off[:, :n], off[:, n:])
    got = moe.int8_gated(c.x, c.scale, c.w, c.w_scale, c.offsets, activation=act, dtype=t)
    check(torch, got, h, rounded(torch, h, before, t), "h")


def test_int8_largest_sums(torch, moe):
    """The longest contraction with every product at its largest: 2^16 x 2^14 fits the int32 sum."""
    k = 65536
    for rows in (1, 65):
        x = torch.full((rows, k), -128, dtype=torch.int8, device="cuda")
        w = torch.full((1, 8, k), -128, dtype=torch.int8, device="cuda")
        w[0, 1::2] = 127
        one = torch.ones(rows, device="cuda")
        got = moe.int8_product(x, one, w, torch.ones(1, 8, device="cuda"), dtype=torch.float32)
        ref = torch.tensor([k * 16384.0, -k * 16256.0] * 4, device="cuda").expand(rows, 8)
        assert torch.equal(got, ref)


# ---- quantising rows ----------------------------------------------------------

def quantize64(torch, x):
    wide = x.double()
    top = wide.abs().amax(1)
    codes = torch.round(wide * 127 / torch.where(top > 0, top, torch.ones_like(top))[:, None])
    return codes.to(torch.int8), top / 127


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 64), (5, 1008), (7, 1024), (2, 1040), (16, 4096), (3, 4112), (33, 14336),
                                    (2, 16384), (3, 20000), (1, 65536), (3, 8), (5, 24), (3, 1032), (4, 4104),
                                    (2, 16392), (1, 65528)])
def test_quantize_rows(torch, moe, rows, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    t = getattr(torch, dtype)
    x = torch.randn(rows, k, generator=gen, device="cuda").to(t)
    x[0, 0] = 5.0
    x[0, 1:8] = 2.5  # exact ties: 63.5
    codes, scale = moe.quantize_rows(x)
    ref, s = quantize64(torch, x)
    assert torch.equal(codes, ref)
    assert ((scale.double() - s).abs() <= E * s).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_value(torch, moe, dtype):
    """Every finite 16-bit value at or below several row maxima, subnormal and largest ones among them."""
    t = getattr(torch, dtype)
    every = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(t)
    every = every[every.isfinite()]
    tops = [torch.finfo(t).max, 1.0, 1.9921875, 3.0, 0.7109375, 1e-3, torch.finfo(t).tiny, torch.finfo(t).tiny * 3,
            torch.finfo(t).tiny / 4, torch.finfo(t).smallest_normal * torch.finfo(t).eps]
    for top in tops:
        top = torch.tensor(top, device="cuda").to(t)
        x = torch.where(every.abs() <= top, every, torch.zeros_like(every))[:65504 // 16 * 16]
        x = torch.cat([x, torch.zeros(-x.numel() % 16, dtype=t, device="cuda")])
        x[0] = top
        codes, scale = moe.quantize_rows(x[None, :])
        ref, s = quantize64(torch, x[None, :])
        assert torch.equal(codes, ref), top
        # half a step of the smallest fp32 subnormal where the scale is one
        assert ((scale.double() - s).abs() <= E * s + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [64, 4096, 8192])
def test_quantize_zero_and_nonfinite_rows(torch, moe, dtype, k):
    x = torch.randn(6, k, device="cuda").to(getattr(torch, dtype))
    x[1] = 0
    x[2, k - 1] = float("nan")
    x[3, 0] = float("inf")
    x[4, k // 2] = float("-inf")
    x[5] = -0.0
    codes, scale = moe.quantize_rows(x)
    ref, s = quantize64(torch, x[:1])
    assert torch.equal(codes[:1], ref) and not codes[1:].any()
    assert scale[1] == 0 and scale[5] == 0 and scale[2:5].isnan().all()
    # such rows' products are NaN, the others' are not
    w = torch.ones(1, 8, k, dtype=torch.int8, device="cuda")
    y = moe.int8_product(codes, scale, w, torch.ones(1, 8, device="cuda"))
    assert y[2:5].isnan().all() and y[[0, 1, 5]].isfinite().all()


# ---- rows outside the groups, strides, infinities --------------------------------

def strided(torch, t, pad, fill):
    """The same matrix with `pad` more elements between its rows (a view)."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


@pytest.mark.parametrize("sizes,n,k", [([5, 0, 9], 72, 208), ([100, 0, 150, 3], 264, 208), ([1500, 0, 700, 3], 520, 4112), ([2000, 1500], 2560, 80)],
                         ids=str)
def test_rows_of_no_group_and_strides(torch, moe, sizes, n, k):
    """Rows before and behind the groups hold NaN and are neither read nor written, nor is the space between rows."""
    bf16, nan = torch.bfloat16, float("nan")
    c = Case(torch, sizes, n, k, bf16, before=3, after=6)
    m = c.member()
    c.x[~m] = nan
    _, x = strided(torch, c.x, 24, nan)
    y, before = c.forward()
    bound = rounded(torch, y, before, bf16)

    def buffers(width, dtype=bf16, pad=8):
        buf = torch.full((c.rows, width + pad), 7.0, dtype=dtype, device="cuda")
        return buf, buf[:, :width]

    def untouched(buf, width):
        assert (buf[~m] == 7.0).all() and (buf[:, width:] == 7.0).all()

    buf, out = buffers(n)
    assert moe.expert_product(x, c.w, c.offsets, out=out) is out
    untouched(buf, n)
    check(torch, out[m], y[m], bound[m], "y")

    dy = c.normal(c.rows, n)
    dy[~m] = nan
    _, dys = strided(torch, dy, 40, nan)
    dx, dw, dx_off, dw_off = grads64(torch, c, dy.double(), torch.zeros(c.rows, n, dtype=torch.float64, device="cuda"))
    buf, got = buffers(k)
    _, got_dw = moe.expert_product_backward(dys, x, c.w, c.offsets, dx=got)
    untouched(buf, k)
    check(torch, got[m], dx[m], rounded(torch, dx, dx_off, bf16)[m], "dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, bf16), "dw")

    g = Case(torch, sizes, n, k, bf16, wide=2, before=3, after=6, seed=1)
    g.x[~m] = nan
    _, gx = strided(torch, g.x, 24, nan)
    y, before = g.forward()
    h, h_before = gated64(torch, "silu", y[:, :n], y[:, n:], before[:, :n], before[:, n:])
    hb, hv = buffers(n)
    kb, kv = buffers(2 * n)
    moe.gated_product(gx, g.w, g.offsets, out=hv, gate_up=kv)
    untouched(hb, n)
    untouched(kb, 2 * n)
    check(torch, hv[m], h[m], rounded(torch, h, h_before, bf16)[m], "h")
    check(torch, kv[m], y[m], rounded(torch, y, before, bf16)[m], "gate_up")
    kv[~m] = nan
    d, off = slopes64(torch, "silu", dy, kv, n, bf16)
    dx, dw, dx_off, dw_off = grads64(torch, g, d, off)
    buf, got = buffers(k)
    _, got_dw = moe.gated_product_backward(dys, kv, gx, g.w, g.offsets, dx=got)
    untouched(buf, k)
    check(torch, got[m], dx[m], rounded(torch, dx, dx_off, bf16)[m], "dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, bf16), "dw")

    # codes: quantise the strided rows (those of no group get scale NaN), then the product leaves them alone
    codes, scale = moe.quantize_rows(x)
    assert scale[~m].isnan().all()
    cb = torch.zeros(c.rows, k + 32, dtype=torch.int8, device="cuda")
    cb[:, :k] = codes
    wq, ws = moe.quantize_rows(c.w.view(-1, k))
    buf, out = buffers(n, torch.float32)
    moe.int8_product(cb[:, :k], scale, wq.view(c.w.shape), ws.view(c.w.shape[:2]), c.offsets, out=out)
    untouched(buf, n)
    ref = torch.zeros(c.rows, n, dtype=torch.float64, device="cuda")
    for e, b, t in c.groups():
        ref[b:t] = (codes[b:t].double() @ wq.view(c.w.shape)[e].double().t().contiguous()) * scale[b:t, None].double() * ws.view(-1, n)[e].double()
    check(torch, out[m], ref[m], rounded(torch, ref, 3 * E * ref.abs(), torch.float32)[m], "int8")


@pytest.mark.parametrize("rows", [5, 300, 5000])
def test_nonfinite_values_stay_in_their_row_and_group(torch, moe, rows):
    c = Case(torch, [rows, rows], 72, 136, torch.bfloat16)
    c.x[1, 5] = float("nan")
    c.x[2, 7] = float("inf")
    y = moe.expert_product(c.x, c.w, c.offsets)
    assert y[1].isnan().all() and not y[2].isfinite().any()
    rest = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    rest[1:3] = False
    assert y[rest].isfinite().all()
    dy = c.normal(c.rows, 72)
    dx, dw = moe.expert_product_backward(dy, c.x, c.w, c.offsets)
    assert dx.isfinite().all()
    assert dw[0, :, 5].isnan().all() and dw[1].isfinite().all()
    keep = [i for i in range(136) if i not in (5, 7)]
    assert dw[0][:, keep].isfinite().all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_extremes(torch, moe, act):
    """Gates far out: the sigmoid saturates without overflow; NaN stays NaN."""
    g = torch.tensor([-1e30, -1e4, -300.0, -88.0, -20.0, -1e-30, 0.0, 1e-30, 20.0, 88.0, 300.0, 1e4, 1e15, float("nan"),
                      -0.0, 1.0], device="cuda").to(torch.bfloat16)
    rows = g.numel()
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = g
    x[:, 1] = 1.0
    w = torch.zeros(1, 16, 8, dtype=torch.bfloat16, device="cuda")
    w[0, :8, 0] = 1.0  # gate = g
    w[0, 8:, 1] = 1.0  # up = 1
    h, gu = moe.gated_product(x, w, activation=act, save=True)
    nan = g.isnan()
    ref, slope, z, _ = act64(torch, act, g.double()[:, None].expand(rows, 8))
    assert h[nan].isnan().all()
    fine = ~nan
    bound = rounded(torch, ref, 2 * E * (8 + 4 * z) * ref.abs(), torch.bfloat16) + 2.0 ** -126  # results below the normal range
    check(torch, h[fine], ref[fine], bound[fine], "h")
    dh = torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda")
    one = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    pick = torch.cat([one, torch.zeros_like(one)])[None].contiguous()  # dx = dg
    dx, _ = moe.gated_product_backward(dh, gu, x, pick, activation=act, need_dw=False)
    inside = fine & (g.abs() <= 1e4)
    slope = torch.where(slope.isnan(), (g.double() > 0).double()[:, None], slope)
    off = 2 * E * (16 + 8 * z) * slope.abs().clamp_max(2) + 2 * E * 16 + 2.0 ** -126
    b = rounded(torch, slope, rounded(torch, slope, off, torch.bfloat16), torch.bfloat16)
    check(torch, dx[inside], slope[inside], b[inside], "dg")


# ---- gradients against differences -------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(torch, moe, act):
    """<dx, v> + <dw, V> against the central difference of L = sum dh h along (v, V), L in 64 bits.
    The gradient sees (g, u) rounded to fp16: dg moves by |dh u act''| du + |dh act'| du for half-steps du."""
    sizes, n, k, t = [70, 0, 33], 72, 136, torch.float16
    c = Case(torch, sizes, n, k, t, wide=2, seed=3)
    dh = c.normal(c.rows, n)
    h, gu = moe.gated_product(c.x, c.w, c.offsets, activation=act, save=True)
    dx, dw = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, activation=act, dw_dtype=torch.float32)
    v = c.normal(c.rows, k).double()
    V = c.normal(*c.w.shape, std=k ** -0.5).double()

    def loss(step):
        total = 0.0
        for e, b, e2 in c.groups():
            y = (c.x[b:e2].double() + step * v[b:e2]) @ (c.w[e].double() + step * V[e]).t().contiguous()
            total = total + (act64(torch, act, y[:, :n])[0] * y[:, n:] * dh[b:e2].double()).sum()
        return total

    step = 1e-5
    difference = (loss(step) - loss(-step)) / (2 * step)
    got = (dx.double() * v).sum() + (dw.double() * V).sum()
    # the kernel's own roundings
    d, off = slopes64(torch, act, dh, gu, n, t)
    y, before = c.forward()
    gap = rounded(torch, y, before, t)
    _, slope, _, _ = act64(torch, act, y[:, :n])
    curve = 1.0  # |act''| is below 1 for both
    g, u = y[:, :n], y[:, n:]
    more_g = dh.double().abs() * (gap[:, n:] * (slope.abs() + curve * gap[:, :n]) + u.abs() * curve * gap[:, :n])
    more_u = dh.double().abs() * 1.13 * gap[:, :n]
    rx, rw, rx_off, rw_off = grads64(torch, c, d, off + torch.cat([more_g, more_u], 1))
    bound = (rounded(torch, rx, rx_off, t) * v.abs()).sum() + (rounded(torch, rw, rw_off, torch.float32) * V.abs()).sum()
    # the difference itself: step^2 / 6 times a third derivative, and 64-bit cancellation
    bound = bound + 1e-4 * got.abs()
    say(f"difference {difference.item():.6f} gradient {got.item():.6f} bound {bound.item():.4f}")
    assert (got - difference).abs() <= bound


# ---- how the calls are used --------------------------------------------------------

def every_call(torch, moe, rows, n, k, seed=0, t=None):
    """(name, function of no arguments returning tensors) for each operator."""
    t = t or torch.bfloat16
    sizes = [rows // 3, 0, rows - rows // 3]
    p = Case(torch, sizes, n, k, t, seed=seed)
    g = Case(torch, sizes, n, k, t, wide=2, seed=seed + 1)
    dy = p.normal(p.rows, n)
    gu = g.normal(g.rows, 2 * n)
    codes, scale = moe.quantize_rows(p.x)
    wq, ws = (a.view(*p.w.shape[:2], *a.shape[1:]) for a in moe.quantize_rows(p.w.view(-1, k)))
    gq, gs = (a.view(*g.w.shape[:2], *a.shape[1:]) for a in moe.quantize_rows(g.w.view(-1, k)))
    torch.cuda.synchronize()
    return [("quantize_rows", lambda **kw: moe.quantize_rows(p.x, **kw)),
            ("int8_product", lambda **kw: moe.int8_product(codes, scale, wq, ws, p.offsets, **kw)),
            ("int8_gated", lambda **kw: moe.int8_gated(codes, scale, gq, gs, p.offsets, **kw)),
            ("expert_product", lambda **kw: moe.expert_product(p.x, p.w, p.offsets, **kw)),
            ("expert_product_backward", lambda **kw: moe.expert_product_backward(dy, p.x, p.w, p.offsets, **kw)),
            ("gated_product", lambda **kw: moe.gated_product(g.x, g.w, g.offsets, save=True, **kw)),
            ("gated_product_backward", lambda **kw: moe.gated_product_backward(dy, gu, g.x, g.w, g.offsets, **kw))]


def tensors(out):
    return list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("rows", [7, 300, 2500])
def test_same_call_same_bits_on_any_stream(torch, moe, rows):
    side = torch.cuda.Stream()
    for name, call in every_call(torch, moe, rows, n=128, k=4096):  # few blocks: split contractions
        first = tensors(call())
        torch.cuda.synchronize()
        other = tensors(call(stream=side))
        with torch.cuda.stream(side):
            inside = tensors(call())
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, inside):
            assert torch.equal(a, b) and torch.equal(a, c), name


def test_inputs_freed_while_another_stream_reads_them(torch, moe):
    """Inputs dropped right after a call on a side stream keep their memory until it is done."""
    side = torch.cuda.Stream()
    w = torch.randn(1, 4096, 4096, device="cuda").to(torch.bfloat16)
    for _ in range(4):
        x = torch.randn(8192, 4096, device="cuda").to(torch.bfloat16)
        ref = moe.expert_product(x, w)
        torch.cuda.synchronize()
        moe.expert_product(x, w, stream=side)  # keeps the side stream busy first
        y = moe.expert_product(x, w, stream=side)
        where = x.data_ptr()
        del x
        other = [torch.full((8192, 4096), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(y, ref), [t.data_ptr() == where for t in other]


@pytest.mark.parametrize("rows", [7, 300, 2500])
def test_captured_calls_replay(torch, moe, rows):
    """Each call captured into a graph with its buffers; replays follow rewritten inputs, with eager work between."""
    for index, (name, call) in enumerate(every_call(torch, moe, rows, n=128, k=4096)):
        expected = [t.clone() for t in tensors(call())]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tensors(call())
        for _ in range(3):
            for t in out:
                t.zero_()
            graph.replay()
            eager = tensors(call())
            torch.cuda.synchronize()
            for a, b, c in zip(out, expected, eager):
                assert torch.equal(a, b) and torch.equal(c, b), name
        del graph


def test_two_graphs_share_a_workspace(torch, moe):
    """Graphs over one workspace, replayed one after the other, keep nothing in it between calls."""
    c = Case(torch, [1000], 256, 8192, torch.bfloat16)
    d = Case(torch, [900], 1024, 8192, torch.bfloat16, seed=1)
    needs = [moe.product_workspace("expert_product", 1000, 256, 8192),
             moe.product_workspace("expert_product", 900, 1024, 8192)]
    assert min(needs) > 0
    ws = torch.empty(max(needs), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(1000, 256, dtype=torch.bfloat16, device="cuda"),
            torch.empty(900, 1024, dtype=torch.bfloat16, device="cuda")]
    refs = [moe.expert_product(c.x, c.w), moe.expert_product(d.x, d.w)]
    torch.cuda.synchronize()
    graphs = []
    for case, out in zip((c, d), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.expert_product(case.x, case.w, out=out, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0)):
        for o in outs:
            o.zero_()
        ws.fill_(0xFF)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])


def test_given_buffers_and_refusals(torch, moe):
    c = Case(torch, [1000], 256, 8192, torch.bfloat16)
    need = moe.product_workspace("expert_product", 1000, 256, 8192)
    with pytest.raises(moe.MoeError) as e:
        moe.expert_product(c.x, c.w, workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    out, ws = torch.empty(1000, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")
    moe.expert_product(c.x, c.w, out=out, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before + 2  # the two above
    with pytest.raises(ValueError, match="w must be"):
        moe.expert_product(c.x, c.w.half())
    with pytest.raises(ValueError, match="must be"):
        moe.expert_product(c.x, c.w[:, :, :4096])
    with pytest.raises(ValueError, match="contiguous"):
        moe.expert_product(c.x, c.w.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        moe.expert_product(c.x.t().contiguous().t(), c.w)
    with pytest.raises(ValueError, match="offsets must be"):
        moe.expert_product(c.x, c.w, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="offsets must be"):
        moe.expert_product(c.x, c.w, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="offsets is on"):
        moe.expert_product(c.x, c.w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="unsupported dtype"):
        moe.expert_product(c.x.double(), c.w.double())
    with pytest.raises(moe.MoeError):
        moe.expert_product(c.x.float(), c.w.float())
    with pytest.raises(moe.MoeError):
        moe.expert_product(c.x[:1].expand(1000, -1), c.w, workspace=ws)  # rows on top of each other
    with pytest.raises(moe.MoeError):
        moe.expert_product(c.x[:, 1:9], c.w[:, :, 1:9].contiguous())    # rows off their alignment
    with pytest.raises(moe.MoeError):
        moe.int8_gated(*moe.quantize_rows(c.x), torch.zeros(1, 16, 8192, dtype=torch.int8, device="cuda"),
                       torch.zeros(1, 16, device="cuda"), dtype=torch.float32)
    torch.cuda.synchronize()


def test_offsets_out_of_order_or_range(torch, moe):
    """Nothing outside the matrices is touched: rows and offsets are clamped (0..100, none, 60..200 of 200 rows)."""
    rows, n, k = 200, 72, 136
    off = torch.tensor([-5, 100, 60, 1 << 30], dtype=torch.int32, device="cuda")
    for scale in (1, 40):  # few rows and tiles
        r = rows * scale
        offsets = torch.where(off == 1 << 30, off, off * scale).to(torch.int32)
        buf = torch.full((r + 20, n), 7.0, dtype=torch.bfloat16, device="cuda")
        x = torch.randn(r, k, device="cuda").to(torch.bfloat16)
        w = torch.randn(3, n, k, device="cuda").to(torch.bfloat16)
        moe.expert_product(x, w, offsets, out=buf[10:-10])
        assert (buf[:10] == 7.0).all() and (buf[-10:] == 7.0).all()
        dxb = torch.full((r + 20, k), 7.0, dtype=torch.bfloat16, device="cuda")
        _, dw = moe.expert_product_backward(buf[10:-10], x, w, offsets, dx=dxb[10:-10])
        assert (dxb[:10] == 7.0).all() and (dxb[-10:] == 7.0).all() and not dw[1].any()
        torch.cuda.synchronize()


def test_no_rows(torch, moe):
    """Calls without rows, and with only empty groups: nothing is written but zero weight gradients."""
    bf16 = torch.bfloat16
    for rows in (0, 5, 200):
        x = torch.zeros(rows, 64, dtype=bf16, device="cuda")
        w = torch.ones(3, 48, 64, dtype=bf16, device="cuda")
        off = torch.full((4,), rows // 2, dtype=torch.int32, device="cuda")
        out = torch.full((rows, 48), 3.0, dtype=bf16, device="cuda")
        moe.expert_product(x, w, off, out=out)
        assert (out == 3.0).all()
        h = torch.full((rows, 24), 3.0, dtype=bf16, device="cuda")
        moe.gated_product(x, w, off, out=h)
        assert (h == 3.0).all()
        dx = torch.full((rows, 64), 3.0, dtype=bf16, device="cuda")
        for dw_dtype in (bf16, torch.float32):
            _, dw = moe.expert_product_backward(out, x, w, off, dx=dx, dw_dtype=dw_dtype)
            assert (dx == 3.0).all() and not dw.any()
        _, dw = moe.gated_product_backward(h, torch.zeros(rows, 48, dtype=bf16, device="cuda"), x, w, off, dx=dx)
        assert (dx == 3.0).all() and not dw.any()
        codes, scale = moe.quantize_rows(x)
        assert codes.shape == (rows, 64) and scale.shape == (rows,)
    assert moe.expert_product(torch.zeros(0, 64, dtype=bf16, device="cuda"), w[0]).shape == (0, 48)


def test_past_32_bits(torch, moe):
    """Row matrices and weights larger than 4 GiB: the last rows and the last group."""
    bf16 = torch.bfloat16
    rows, k, n = 620_000, 4096, 16
    x = torch.zeros(rows, k, dtype=bf16, device="cuda")
    tail = torch.randn(300, k, device="cuda").to(bf16)
    x[-300:] = tail
    w = (torch.randn(2, n, k, device="cuda") / 64).to(bf16)
    off = torch.tensor([0, rows - 300, rows], dtype=torch.int32, device="cuda")
    y = moe.expert_product(x, w, off)
    ref = tail.double() @ w[1].double().t().contiguous()
    bound = rounded(torch, ref, 2 * k * E * (tail.double().abs() @ w[1].double().abs().t().contiguous()), bf16)
    check(torch, y[-300:], ref, bound, "last rows")
    assert not y[:-300].any()
    codes, scale = moe.quantize_rows(x)
    ref_codes, _ = quantize64(torch, tail)
    assert torch.equal(codes[-300:], ref_codes) and not codes[: rows - 300].any()
    dy = torch.zeros(rows, n, dtype=bf16, device="cuda")
    dy[-300:] = torch.randn(300, n, device="cuda").to(bf16)
    dx, dw = moe.expert_product_backward(dy, x, w, off)
    ref = dy[-300:].double().t().contiguous() @ tail.double()
    bound = 2 * 300 * E * (dy[-300:].double().abs().t().contiguous() @ tail.double().abs())
    check(torch, dw[1], ref, rounded(torch, ref, bound, bf16), "dw")
    assert not dw[0].any() and not dx[:-300].any() and dx[-300:].any()
    del x, codes, dx, y
    groups, n, k = 40, 8192, 8192  # 5.4 GB of weights
    w = torch.zeros(groups, n, k, dtype=bf16, device="cuda")
    w[-1] = (torch.randn(n, k, device="cuda") / 90).to(bf16)
    for last in (3, 100, 2000):
        x = torch.randn(last + groups - 1, k, device="cuda").to(bf16)
        off = torch.tensor(list(range(groups)) + [last + groups - 1], dtype=torch.int32, device="cuda")
        ref = x[-last:].double() @ w[-1].double().t().contiguous()
        bound = 2 * k * E * (x[-last:].double().abs() @ w[-1].double().abs().t().contiguous())
        y = moe.expert_product(x, w, off)
        check(torch, y[-last:], ref, rounded(torch, ref, bound, bf16), "last group")
        assert not y[:-last].any()


def test_with_the_layer(torch, moe):
    """The layer's routing feeds the products: gather, quantise-free 16-bit block and int8 block, weighted sum.
    The 16-bit block computes what the layer computes from the same dequantised weights."""
    import synth
    from gpu_util import GpuLayer, bf16_bits_to_f64
    case = synth.make_case("tiny_q8")
    s, w = case.shape, case.weights
    gpu = GpuLayer(s, w)
    res = gpu.run(case.hidden)
    T, top = s.T, s.top_k
    bf16 = torch.bfloat16

    def dense(codes, scale, zero):
        q = torch.from_numpy(codes.astype(np.float32))
        sc = torch.from_numpy(scale.view(np.float16).astype(np.float32))
        z = torch.from_numpy(zero.view(np.float16).astype(np.float32))
        return ((q - z[..., None]) * sc[..., None])[torch.from_numpy(w.slot_table[: s.num_experts]).long()]

    gate, up, down = (dense(getattr(w, f"w_{m}"), getattr(w, f"s_{m}"), getattr(w, f"z_{m}")) for m in ("gate", "up", "down"))
    gate_up = torch.cat([gate, up], 1).to(bf16).cuda().contiguous()
    down = down.to(bf16).cuda().contiguous()
    x = gpu.hidden(case.hidden)
    perm = torch.from_numpy(res["perm"]).long().cuda()
    offsets = torch.from_numpy(res["offsets"]).cuda()
    weight = torch.from_numpy(res["topk_w"]).cuda().reshape(-1)[perm]
    rows = x[perm // top]
    h, gu = moe.gated_product(rows, gate_up, offsets, save=True)
    y = moe.expert_product(h, down, offsets)
    out = torch.zeros(T, s.d_model, device="cuda").index_add_(0, perm // top, y.float() * weight[:, None])
    ref = torch.from_numpy(res["out"]).cuda()
    rms = ref.square().mean().sqrt()
    # the layer's own parity bound, 2e-2, plus the weights' rounding to bf16 here (2^-8 each of three factors)
    worst = ((out.double() - ref).abs() / ref.abs().clamp_min(rms)).max()
    say(f"16-bit block against the layer: {worst.item():.4f}")
    assert worst <= 2e-2 + 3 * 2.0 ** -8

    # the gradients of the block chained through both products, against 64-bit autograd of the formula
    dout = torch.randn(T, s.d_model, device="cuda").to(bf16)
    dy = (dout.float()[perm // top] * weight[:, None]).to(bf16)
    dh, ddown = moe.expert_product_backward(dy, h, down, offsets)
    dx, dgu = moe.gated_product_backward(dh, gu, rows, gate_up, offsets)
    ends = res["offsets"].tolist()
    r64, w64, d64 = (t.double().requires_grad_() for t in (rows, gate_up, down))
    parts = []
    for e in range(s.num_experts):
        z = r64[ends[e]:ends[e + 1]] @ w64[e].t()
        g, u = z.split(s.d_ff, 1)
        parts.append((torch.sigmoid(g) * g * u) @ d64[e].t())
    torch.cat(parts).backward(dy.double())
    for name, got, want in (("dx", dx, r64.grad), ("dw gate_up", dgu, w64.grad), ("dw down", ddown, d64.grad)):
        off = (got.double() - want).norm() / want.norm()
        # h, dh, (g, u) and (dg, du) are each rounded once (2^-8 at most), as is the result
        say(f"{name}: {off.item():.5f}")
        assert off <= 5 * 2.0 ** -8, name

    # 8-bit block: codes of the rows, the gated product, codes of h, the down product
    gq, gs = moe.quantize_rows(gate_up.view(-1, s.d_model))
    dq, ds = moe.quantize_rows(down.view(-1, s.d_ff))
    gq, gs = gq.view(gate_up.shape), gs.view(gate_up.shape[:2])
    dq, ds = dq.view(down.shape), ds.view(down.shape[:2])
    h8 = moe.int8_gated(*moe.quantize_rows(rows), gq, gs, offsets)
    y8 = moe.int8_product(*moe.quantize_rows(h8), dq, ds, offsets)
    # exactly the block on the values that the codes stand for, up to bf16 roundings of h8 and y8
    xq, xs = moe.quantize_rows(rows)
    hq, hs = moe.quantize_rows(h8)
    for e in range(s.num_experts):
        b, t = ends[e], ends[e + 1]
        z = (xq[b:t].double() * xs[b:t, None].double()) @ (gq[e].double() * gs[e][:, None].double()).t().contiguous()
        g, u = z.split(s.d_ff, 1)
        hr = torch.sigmoid(g) * g * u
        assert ((h8[b:t].double() - hr).abs() <= hr.abs() * 2.0 ** -8 * 1.01 + 1e-12).all()
        yr = (hq[b:t].double() * hs[b:t, None].double()) @ (dq[e].double() * ds[e][:, None].double()).t().contiguous()
        assert ((y8[b:t].double() - yr).abs() <= yr.abs() * 2.0 ** -8 * 1.01 + 1e-12).all()
