"""The products in 8-bit floating point on the GPU against plain 64-bit ones.

Bounds, per element, from the roundings alone (u = half a step of the output's
type relative to the value, 2^-8 bf16, 2^-11 fp16, 2^-24 fp32; e = 2^-24):
  sums     the matrix cores cut each of a block's products off at 2^-13 of
           the largest (measured, one product beside another: at the power of
           two at or below it, whatever else is added), no larger than the
           product of both operands' largest: 128 2^-13 max |x| max |w|, summed
           over the blocks.  Then 128 additions, each off by at most one step
           (2e: they may truncate) of a partial sum no larger than the block's
           S_b = sum |x w|: 256 e S_b.  The scales' product and its product
           with the block round to e each, joined by FMA: 2e S_b.  The
           additions of blocks, of the waves' or the parts' sums (16 at most):
           e of a partial sum no larger than S each.  In all
           (258 + blocks + 16) e S, S = sum |x w| with the scales, and the cut
  act(g)   as for the products in 16 bits: A = 2e (8 + 4 |z|) |act(g)|; the
           error d of g moves act(g) by at most 1.13 d
  codes    e4m3 of the exact quotient 448 x / a: equal.  The gated block's
           slopes are known within a bound d; their codes then lie between
           those of x - d and x + d, with the largest magnitude as uncertain
  output   u |value|, and half of the smallest subnormal (2^-25 in fp16,
           2^-134 in bf16: below 2^-126 its values lie 2^-133 apart)
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say
from test_gpu_products import E, act64, check, gated64
from test_gpu_products import rounded as rounded_normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


TYPES = ["bfloat16", "float16"]


def rounded(torch, value, before, dtype):
    """Bound of the output: the error before rounding, plus the rounding."""
    return rounded_normal(torch, value, before, dtype) + (2.0 ** -134 if dtype == torch.bfloat16 else 0.0)


def blocks(n):
    return (n + 127) // 128


def spread(scale, k):
    """Scales of blocks -> of values, along the last dimension."""
    return scale.double().repeat_interleave(128, dim=-1)[..., :k]


def tops(x):
    """The largest magnitude of each 128 along the last dimension."""
    whole = x.new_zeros(x.shape[0], blocks(x.shape[1]) * 128)
    whole[:, :x.shape[1]] = x.abs()
    return whole.view(x.shape[0], -1, 128).amax(2)


class Case:
    """Codes of one grouped product: `contract` is the length of the sums over `halves` matrices of a group;
    `before` and `after` rows belong to no group."""

    def __init__(self, torch, sizes, n, k, gated=False, backward=False, before=0, after=0, seed=0, wild=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.sizes, self.n, self.k, self.gen = torch, sizes, n, k, gen
        self.rows = before + sum(sizes) + after
        self.ends = [before]
        for s in sizes:
            self.ends.append(self.ends[-1] + s)
        self.offsets = torch.tensor(self.ends, dtype=torch.int32, device="cuda")
        self.halves = 2 if gated else 1
        width = n if backward else k
        self.codes, self.scale = self.draw((self.rows, width), (blocks(width), self.rows), wild)
        matrix = (len(sizes),) + ((2,) if gated else ())
        self.w, self.w_scale = self.draw((*matrix, n, k), (*matrix, blocks(n), blocks(k)), wild)
        if not wild:
            self.w_scale *= width ** -0.5
        self.width = width

    def draw(self, shape, scales, wild):
        """Every finite code alike, or normal ones; scales over a factor of some ten (wild: 2^40)."""
        torch = self.torch
        if wild:
            codes = torch.randint(0, 0x7F, shape, generator=self.gen, device="cuda", dtype=torch.uint8)
            codes |= torch.randint(0, 2, shape, generator=self.gen, device="cuda", dtype=torch.uint8) << 7
            codes = codes.view(torch.float8_e4m3fn)
            scale = torch.exp2(torch.randn(scales, generator=self.gen, device="cuda") * 5)
        else:
            codes = (torch.randn(shape, generator=self.gen, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            scale = torch.exp(torch.randn(scales, generator=self.gen, device="cuda") * 0.5) / 100
        return codes, scale

    def groups(self):
        return [(e, self.ends[e], self.ends[e + 1]) for e in range(len(self.sizes)) if self.sizes[e]]

    def x64(self):
        return self.codes.double() * spread(self.scale.t(), self.width)

    def w64(self, e):
        """[halves n, k]"""
        s = spread(self.w_scale[e], self.k).repeat_interleave(128, dim=-2)[..., :self.n, :]
        return (self.w[e].double() * s).reshape(self.halves * self.n, self.k)

    def product(self, x=None, backward=False):
        """(y, bound of its sums) in 64 bits; rows of no group are zero."""
        torch = self.torch
        x = self.x64() if x is None else x
        width = x.shape[1]
        total = self.halves * blocks(self.n) if backward else blocks(self.k)
        y = torch.zeros(self.rows, self.k if backward else self.halves * self.n, dtype=torch.float64, device="cuda")
        s = torch.zeros_like(y)
        for e, b, t in self.groups():
            w = self.w64(e)
            w = w if backward else w.t().contiguous()
            y[b:t] = x[b:t] @ w
            s[b:t] = (258 + total + 16) * E * (x[b:t].abs() @ w.abs())
            half = self.n if backward else self.k
            for at in range(0, width, half):  # the blocks of either half
                s[b:t] += 2.0 ** -6 * (tops(x[b:t, at:at + half]) @ tops(w[at:at + half].t()).t().contiguous())
        return y, s


# sizes, n, k: one row to several tiles, empty groups, partial tiles, widths that end inside a 16-column tile's
# block of 128 and inside a 64-byte step
FEW = [([1], 16, 16), ([1], 64, 4096), ([3], 1008, 80), ([16], 48, 144), ([17], 32, 64), ([33], 272, 2064),
       ([64], 128, 528), ([0, 1, 0, 5, 16, 0, 7], 80, 208), ([20, 0, 44], 144, 336), ([2], 16, 128), ([1], 4096, 2048),
       ([7], 256, 640)]
TILES = [([65], 16, 16), ([129], 144, 80), ([200], 1008, 1424), ([0, 70, 0, 1, 128, 255, 0], 272, 208),
         ([256, 300], 128, 64), ([1000], 400, 464), ([3, 130, 67], 1008, 2064)]
MANY = [([150] + [0] * 8, 16, 16), ([0, 70, 0, 1, 128, 255, 0, 0, 0, 0], 272, 208), ([1000] + [0] * 8, 400, 464),
        ([0] * 8 + [200], 1008, 1424), ([3, 130, 67] + [0] * 7, 1008, 2064), ([0, 300] + [0] * 8, 272, 8208),
        ([0] * 20 + [700] + [3] * 30 + [0] * 13, 272, 80), ([1, 150] + [7] * 14, 1040, 528)]
# 128-wide tiles whole and split, 256-wide ones with the last round's remainder split
BIG = [([3700], 4096, 80), ([500, 0, 1, 1255, 129, 1100], 1008, 2064), ([2049], 528, 4112), ([4096], 4096, 80),
       ([511, 0, 1300, 257, 700, 130], 2576, 144), ([3000, 1, 900], 4112, 4112)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + MANY + BIG, ids=str)
def test_fp8_product(torch, moe, sizes, n, k, dtype):
    say(f"fp8_product {sizes} {n} {k} {dtype}")
    c = Case(torch, sizes, n, k)
    y, s = c.product()
    got = moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, c.offsets, dtype=getattr(torch, dtype))
    check(torch, got, y, rounded(torch, y, s, getattr(torch, dtype)), "y")


@pytest.mark.parametrize("sizes,n,k", [FEW[5], FEW[7], TILES[3], MANY[4], BIG[1]], ids=str)
def test_fp8_every_code_and_scale(torch, moe, sizes, n, k):
    """Codes of every finite value, subnormal ones among them, and scales over many powers of two."""
    say(f"fp8 every code {sizes} {n} {k}")
    c = Case(torch, sizes, n, k, wild=True)
    y, s = c.product()
    got = moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, c.offsets, dtype=torch.bfloat16)
    check(torch, got, y, rounded(torch, y, s, torch.bfloat16), "y")
    c = Case(torch, sizes, n, k, backward=True, wild=True)
    y, s = c.product(backward=True)
    got = moe.fp8_product_backward(c.codes, c.scale, c.w, c.w_scale, c.offsets, dtype=torch.bfloat16)
    check(torch, got, y, rounded(torch, y, s, torch.bfloat16), "dx")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + MANY + BIG[1:], ids=str)
def test_fp8_gated(torch, moe, sizes, n, k, dtype, act):
    say(f"fp8_gated {sizes} {n} {k} {dtype} {act}")
    t = getattr(torch, dtype)
    c = Case(torch, sizes, n, k, gated=True)
    y, s = c.product()
    h, before = gated64(torch, act, y[:, :n], y[:, n:], s[:, :n], s[:, n:])
    got, gu = moe.fp8_gated(c.codes, c.scale, c.w, c.w_scale, c.offsets, activation=act, save=True, dtype=t)
    check(torch, got, h, rounded(torch, h, before, t), "h")
    check(torch, gu, y, rounded(torch, y, s, t), "gate_up")
    alone = moe.fp8_gated(c.codes, c.scale, c.w, c.w_scale, c.offsets, activation=act, dtype=t)
    assert torch.equal(alone, got)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + BIG, ids=str)
def test_fp8_product_backward(torch, moe, sizes, n, k, dtype):
    say(f"fp8_product_backward {sizes} {n} {k} {dtype}")
    c = Case(torch, sizes, n, k, backward=True)
    dx, s = c.product(backward=True)
    got = moe.fp8_product_backward(c.codes, c.scale, c.w, c.w_scale, c.offsets, dtype=getattr(torch, dtype))
    check(torch, got, dx, rounded(torch, dx, s, getattr(torch, dtype)), "dx")


def e4m3_64(torch, q):
    """e4m3 of 64-bit values, ties to even, as 64-bit values (clamped at the largest)."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(q / step) * step).clamp(-448, 448)


def slopes_codes64(torch, x, off):
    """What the codes of x (within off) stand for, and how far the kernel's may be from that."""
    rows, n = x.shape
    pad = blocks(n) * 128 - n
    x = torch.nn.functional.pad(x, (0, pad)).view(rows, -1, 128)
    off = torch.nn.functional.pad(off, (0, pad)).view(rows, -1, 128)
    top = x.abs().amax(2, keepdim=True)
    top_off = off.amax(2, keepdim=True)  # the largest magnitude moves by no more than the largest of these
    safe = torch.where(top > 0, top, torch.ones_like(top))
    q = x * 448 / safe
    q_off = off * 448 / safe + q.abs() * (top_off / safe) * 1.01 + q.abs() * 4 * E
    value = e4m3_64(torch, q)
    far = torch.maximum((e4m3_64(torch, q - q_off) - value).abs(), (e4m3_64(torch, q + q_off) - value).abs())
    scale = safe / 448
    moved = far * scale * (1 + 1e-3) + value.abs() * scale * (top_off / safe + 2 * E)
    return (value * scale).view(rows, -1)[:, :n], moved.view(rows, -1)[:, :n]


def slopes64(torch, act, dh, gu, n):
    """(dg, du) from the saved (g, u), and how far the kernel's are before their rounding."""
    g, u, d = gu[:, :n].double(), gu[:, n:].double(), dh.double()
    a, slope, z, curve = act64(torch, act, g)
    s = slope - curve * torch.sign(g)  # the sigmoid
    dg, du = d * u * slope, d * a
    dg_off = (d * u).abs() * 2 * E * (16 + 8 * z) * (s.abs() + curve) + 4 * E * dg.abs()
    du_off = d.abs() * 2 * E * (8 + 4 * z) * a.abs() + 2 * E * du.abs()
    return dg, du, dg_off, du_off


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", FEW + TILES + BIG[1:], ids=str)
def test_fp8_gated_backward(torch, moe, sizes, n, k, dtype, act):
    say(f"fp8_gated_backward {sizes} {n} {k} {dtype} {act}")
    t = getattr(torch, dtype)
    c = Case(torch, sizes, n, k, gated=True)
    dh = torch.randn(c.rows, n, generator=c.gen, device="cuda").to(t)
    gu = (torch.randn(c.rows, 2 * n, generator=c.gen, device="cuda") * 2).to(t)
    dg, du, dg_off, du_off = slopes64(torch, act, dh, gu, n)
    (xg, mg), (xu, mu) = slopes_codes64(torch, dg, dg_off), slopes_codes64(torch, du, du_off)
    x, moved = torch.cat([xg, xu], 1), torch.cat([mg, mu], 1)
    dx, _ = c.product(x, backward=True)
    _, far_s = c.product(x.abs() + moved, backward=True)  # bounds of the codes that the kernel may have
    m = torch.zeros_like(dx)
    for e, b, t0 in c.groups():
        m[b:t0] = moved[b:t0] @ c.w64(e).abs()
    got, slopes = moe.fp8_gated_backward(dh, gu, c.w, c.w_scale, c.offsets, activation=act)
    check(torch, got, dx, rounded(torch, dx, m + far_s, t), "dx")
    ref, off = torch.cat([dg, du], 1), torch.cat([dg_off, du_off], 1)
    check(torch, slopes, ref, rounded(torch, ref, off, t), "slopes")
    again, none = moe.fp8_gated_backward(dh, gu, c.w, c.w_scale, c.offsets, activation=act, need_slopes=False)
    assert none is None and torch.equal(again, got)
    none, again = moe.fp8_gated_backward(dh, gu, c.w, c.w_scale, c.offsets, activation=act, need_dx=False)
    assert none is None and torch.equal(again, slopes)


# ---- quantising ----------------------------------------------------------------

def blocks64(torch, x):
    """Codes (as values) and scales of 128 values of a row, from the exact quotients."""
    rows, k = x.shape
    wide = torch.nn.functional.pad(x.double(), (0, blocks(k) * 128 - k)).view(rows, -1, 128)
    top = wide.abs().amax(2, keepdim=True)
    codes = e4m3_64(torch, wide * 448 / torch.where(top > 0, top, torch.ones_like(top)))
    return codes.view(rows, -1)[:, :k], (top[..., 0] / 448).t()


def tiles64(torch, x):
    n, k = x.shape[-2:]
    wide = torch.nn.functional.pad(x.double(), (0, blocks(k) * 128 - k, 0, blocks(n) * 128 - n))
    wide = wide.view(*x.shape[:-2], blocks(n), 128, blocks(k), 128)
    top = wide.abs().amax((-3, -1), keepdim=True)
    codes = e4m3_64(torch, wide * 448 / torch.where(top > 0, top, torch.ones_like(top)))
    return codes.view(*x.shape[:-2], blocks(n) * 128, -1)[..., :n, :k], top[..., 0, :, 0] / 448


def near(scale, s):
    # half a step of the smallest fp32 subnormal where the scale is one
    return ((scale.double() - s).abs() <= E * s + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 64), (5, 1008), (7, 1024), (2, 1040), (16, 4096), (17, 4112), (33, 14336),
                                    (2, 16384), (3, 20000), (1, 65536), (15, 128), (31, 144), (4, 512), (5, 528)])
def test_quantize_blocks(torch, moe, rows, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    t = getattr(torch, dtype)
    x = (torch.randn(rows, k, generator=gen, device="cuda") * torch.exp(torch.randn(rows, k, generator=gen, device="cuda"))).to(t)
    x[0, 0] = 28.0  # quotients 16 x: ties of every kind
    x[0, 1:8] = torch.tensor([1.0625, 1.1875, 0.53125, 0.59375, 17.0 / 16384, 3.0 / 32768, 1.0 / 32768], device="cuda").to(t)
    codes, scale = moe.quantize_blocks(x)
    ref, s = blocks64(torch, x)
    assert codes.dtype == torch.float8_e4m3fn and scale.shape == (blocks(k), rows)
    assert torch.equal(codes.double(), ref)
    assert near(scale, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_blocks_every_value(torch, moe, dtype):
    """Every finite 16-bit value at or below several largest ones, subnormal and largest ones among them."""
    t = getattr(torch, dtype)
    every = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(t)
    every = every[every.isfinite()]
    tops = [torch.finfo(t).max, 1.0, 1.9921875, 3.0, 0.7109375, 1e-3, torch.finfo(t).tiny, torch.finfo(t).tiny * 3,
            torch.finfo(t).tiny / 4, torch.finfo(t).smallest_normal * torch.finfo(t).eps]
    for top in tops:
        top = torch.tensor(top, device="cuda").to(t)
        x = torch.where(every.abs() <= top, every, torch.zeros_like(every))
        x = torch.nn.functional.pad(x, (0, -x.numel() % 127)).view(-1, 127)
        x = torch.cat([top.expand(x.shape[0], 1), x], 1)
        codes, scale = moe.quantize_blocks(x)
        ref, s = blocks64(torch, x)
        assert torch.equal(codes.double(), ref), top
        assert near(scale, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (144, 400), (3, 272, 144), (2, 2, 400, 1040), (1, 1008, 4112), (1, 48), (84, 144),
                                   (3, 131, 272)])
def test_quantize_tiles(torch, moe, shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    t = getattr(torch, dtype)
    x = (torch.randn(shape, generator=gen, device="cuda") * torch.exp(torch.randn(shape, generator=gen, device="cuda"))).to(t)
    codes, scale = moe.quantize_blocks(x, tiles=True)
    ref, s = tiles64(torch, x)
    assert codes.shape == x.shape and scale.shape == s.shape
    assert torch.equal(codes.double(), ref)
    assert near(scale, s)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_zero_and_nonfinite_blocks(torch, moe, dtype, tiles):
    """An infinity or NaN takes its own block with it and no other."""
    x = torch.randn(256, 400, device="cuda").to(getattr(torch, dtype))
    clean, clean_scale = moe.quantize_blocks(x, tiles=tiles)
    x[:, 128:256] = 0
    x[3, 5] = float("nan")
    x[130, 300] = float("-inf")
    codes, scale = moe.quantize_blocks(x, tiles=tiles)
    if tiles:
        bad = torch.tensor([[1, 0, 0, 0], [0, 0, 1, 0]], device="cuda", dtype=torch.bool)
        per_value = bad.repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :400]
    else:
        bad = torch.zeros(4, 256, device="cuda", dtype=torch.bool)
        bad[0, 3] = bad[2, 130] = True
        per_value = bad.t().repeat_interleave(128, 1)[:, :400]
    assert torch.equal(scale.isnan(), bad)
    zero = scale[:, 1] if tiles else scale[1]
    assert not zero.any()
    per_value = per_value.clone()
    per_value[:, 128:256] = True
    assert not codes.view(torch.uint8)[per_value].any()
    assert torch.equal(codes.view(torch.uint8)[~per_value], clean.view(torch.uint8)[~per_value])
