"""The grouped products on the paths that their sizes, offsets and callers choose:
256-wide blocks, split contractions, many groups, replays with other inputs,
rows of no group, gradients past the 16-bit range.

The bounds are those of test_gpu_products.py.  One error is not listed there: the
sigmoid's exponential t is taken of an argument lifted by 64, whose rounding
(2^-19 for |z| < 22) moves t by up to 2^-19 ln 2 = 22 e (e = 2^-24), and the
sigmoid s of a negative z by 22 (1 - s) e.  With at most 4 e for the exponential,
the reciprocal and the products and |z| e for the rounding of log2(e) that is
15 e at z = 0, 21 e at z = -1, 26 e at z = -2 and less than (26 + |z|) e beyond:
inside the bound there, 2e (8 + 4 |z|) = 16 e, 24 e, 32 e, ..."""

import pytest

from gpu_util import say
from test_gpu_products import (E, TYPES, Case, check, gated64, grads64, half_step, int_case, rounded, slopes64,
                               tensors)
from test_gpu_products import moe, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

WIDE_TILE = 256 * 256 * 4  # bytes of one part's raw sums


def sentinel(torch, need):
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)
    return ws


def touched(ws):
    return bool((ws != 0xA5).any())


# ---- 256-wide blocks in codes, and their split contractions ------------------------

# the last one's remaining tiles are split (64 stages of 128 codes)
WIDE = [([4096], 4096, 64), ([511, 0, 1300, 257, 700, 130], 2568, 128), ([3000, 1, 900], 4104, 4096),
        ([2056, 1, 0, 321, 64, 449, 128], 2056, 272), ([3000, 1, 900], 4104, 8192)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", WIDE, ids=str)
def test_int8_gated_wide_blocks(torch, moe, sizes, n, k, dtype, act):
    say(f"int8_gated {sizes} {n} {k} {dtype} {act}")
    c, y = int_case(torch, sizes, n, k, 2)
    t = getattr(torch, dtype)
    off = 3 * E * y.abs()
    h, before = gated64(torch, act, y[:, :n], y[:, n:], off[:, :n], off[:, n:])
    need = moe.product_workspace("int8_gated", c.rows, n, k, len(sizes))
    ws = sentinel(torch, max(need, 1))
    got = moe.int8_gated(c.x, c.scale, c.w, c.w_scale, c.offsets, activation=act, dtype=t, workspace=ws)
    check(torch, got, h, rounded(torch, h, before, t), "h")
    assert need % WIDE_TILE == 0 and touched(ws) == (k == 8192)


@pytest.mark.parametrize("dtype", TYPES + ["float32"])
def test_int8_product_wide_split(torch, moe, dtype):
    sizes, n, k = WIDE[-1]
    say(f"int8_product {sizes} {n} {k} {dtype}")
    c, y = int_case(torch, sizes, n, k, 1)
    t = getattr(torch, dtype)
    ws = sentinel(torch, moe.product_workspace("int8_product", c.rows, n, k, len(sizes)))
    assert ws.numel() == 256 * WIDE_TILE
    got = moe.int8_product(c.x, c.scale, c.w, c.w_scale, c.offsets, dtype=t, workspace=ws)
    check(torch, got, y, rounded(torch, y, 3 * E * y.abs(), t), "y")
    assert touched(ws)


def test_int8_largest_sums_in_tiles(torch, moe):
    """2^16 products of 2^14, with more rows than the streaming kernel takes; parts of the sum are joined."""
    k, rows = 65536, 3500
    x = torch.full((rows, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, 8, k), -128, dtype=torch.int8, device="cuda")
    w[0, 1::2] = 127
    ws = sentinel(torch, moe.product_workspace("int8_product", rows, 8, k))
    got = moe.int8_product(x, torch.ones(rows, device="cuda"), w, torch.ones(1, 8, device="cuda"),
                           dtype=torch.float32, workspace=ws)
    assert torch.equal(got, torch.tensor([k * 16384.0, -k * 16256.0] * 4, device="cuda").expand(rows, 8))
    assert touched(ws)


# ---- many groups ----------------------------------------------------------------------

# more than 64 groups: streaming blocks, 128-wide tiles, 256-wide tiles
CROWDS = [([(5 * e) % 7 for e in range(256)], 72, 208), ([(37 * e) % 61 for e in range(200)], 264, 208),
          ([0] * 130 + [400, 1, 0, 3500] + [0] * 60 + [9] * 62, 136, 80),
          ([150 + (29 * e) % 120 for e in range(100)], 520, 144)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", CROWDS, ids=["256 streaming", "200 small", "256 uneven", "100 wide"])
def test_many_groups(torch, moe, sizes, n, k, dtype):
    say(f"many groups: {len(sizes)} {sum(sizes)} {n} {k} {dtype}")
    t = getattr(torch, dtype)
    c = Case(torch, sizes, n, k, t)
    y, before = c.forward()
    check(torch, moe.expert_product(c.x, c.w, c.offsets), y, rounded(torch, y, before, t), "y")
    dy = c.normal(c.rows, n)
    dx, dw, dx_off, dw_off = grads64(torch, c, dy.double(), torch.zeros(c.rows, n, dtype=torch.float64, device="cuda"))
    got_dx, got_dw = moe.expert_product_backward(dy, c.x, c.w, c.offsets)
    check(torch, got_dx, dx, rounded(torch, dx, dx_off, t), "dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, t), "dw")

    g = Case(torch, sizes, n, k, t, wide=2, seed=1)
    y, before = g.forward()
    h, h_before = gated64(torch, "silu", y[:, :n], y[:, n:], before[:, :n], before[:, n:])
    got, gu = moe.gated_product(g.x, g.w, g.offsets, save=True)
    check(torch, got, h, rounded(torch, h, h_before, t), "h")
    check(torch, gu, y, rounded(torch, y, before, t), "gate_up")
    d, off = slopes64(torch, "silu", dy, gu, n, t)
    dx, dw, dx_off, dw_off = grads64(torch, g, d, off)
    got_dx, got_dw = moe.gated_product_backward(dy, gu, g.x, g.w, g.offsets)
    check(torch, got_dx, dx, rounded(torch, dx, dx_off, t), "gated dx")
    check(torch, got_dw, dw, rounded(torch, dw, dw_off, t), "gated dw")

    i, y = int_case(torch, sizes, n, k, 1)
    got = moe.int8_product(i.x, i.scale, i.w, i.w_scale, i.offsets, dtype=t)
    check(torch, got, y, rounded(torch, y, 3 * E * y.abs(), t), "int8 y")
    i, y = int_case(torch, sizes, n, k, 2)
    off = 3 * E * y.abs()
    h, before = gated64(torch, "gelu", y[:, :n], y[:, n:], off[:, :n], off[:, n:])
    got = moe.int8_gated(i.x, i.scale, i.w, i.w_scale, i.offsets, activation="gelu", dtype=t)
    check(torch, got, h, rounded(torch, h, before, t), "int8 h")


# ---- infinities, NaN and bad offsets in the forward tiles -----------------------------------

@pytest.mark.parametrize("rows,n,k", [(700, 1544, 144), (700, 1544, 8208), (5000, 1032, 144), (3000, 4104, 8208)], ids=str)
def test_nonfinite_values_stay_in_their_row_in_tiles(torch, moe, rows, n, k):
    """128- and 256-wide blocks, whole and split.  A row's infinity or NaN reaches no other row."""
    sizes = [rows, 0, 900]
    split = k > 8000
    need = moe.product_workspace("expert_product", rows + 900, n, k, 3)
    assert (need > 0) == split
    c = Case(torch, sizes, n, k, torch.bfloat16)
    bad = torch.tensor([1, 2, rows - 1, rows + 5], device="cuda")
    c.x[1, 5] = float("nan")
    c.x[2, 7] = float("inf")
    c.x[rows - 1, k - 1] = float("nan")
    c.x[rows + 5, 0] = float("-inf")
    rest = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    rest[bad] = False
    ws = sentinel(torch, max(need, 1))
    y = moe.expert_product(c.x, c.w, c.offsets, workspace=ws)
    assert touched(ws) == split
    assert y[[1, rows - 1]].isnan().all() and not y[bad].isfinite().any() and y[rest].isfinite().all()
    g = Case(torch, sizes, n, k, torch.bfloat16, wide=2)
    h, gu = moe.gated_product(c.x, g.w, g.offsets, save=True)
    assert h[[1, rows - 1]].isnan().all() and h[rest].isfinite().all() and gu[rest].isfinite().all()
    codes, scale = moe.quantize_rows(c.x)
    wq, w_scale = (a.view(*c.w.shape[:2], *a.shape[1:]) for a in moe.quantize_rows(c.w.view(-1, k)))
    y = moe.int8_product(codes, scale, wq, w_scale, c.offsets)
    assert y[bad].isnan().all() and y[rest].isfinite().all()


def test_offsets_out_of_order_in_tiles(torch, moe):
    """Offsets whose groups overlap and make more row tiles than the grids hold: every call stays inside its matrices."""
    n, k = 1032, 144
    bf16 = torch.bfloat16
    for s in (10, 40):  # 128- and 256-wide blocks
        r = 200 * s
        offsets = torch.tensor([-5, 100 * s, 60 * s, 1 << 30], dtype=torch.int32, device="cuda")
        x = torch.randn(r, k, device="cuda").to(bf16)
        w = torch.randn(3, n, k, device="cuda").to(bf16)
        gw = torch.randn(3, 2 * n, k, device="cuda").to(bf16)
        codes, scale = moe.quantize_rows(x)
        wq, ws = (a.view(3, n, *a.shape[1:]) for a in moe.quantize_rows(w.view(-1, k)))
        gq, gs = (a.view(3, 2 * n, *a.shape[1:]) for a in moe.quantize_rows(gw.view(-1, k)))

        def guarded(width, dtype=bf16):
            buf = torch.full((r + 20, width), 7.0, dtype=dtype, device="cuda")
            return buf, buf[10:-10]

        def intact(buf):
            return bool((buf[:10] == 7.0).all() and (buf[-10:] == 7.0).all())

        ob, out = guarded(n)
        moe.expert_product(x, w, offsets, out=out)
        hb, h = guarded(n)
        gb, gu = guarded(2 * n)
        moe.gated_product(x, gw, offsets, out=h, gate_up=gu)
        ib, i8 = guarded(n, torch.float32)
        moe.int8_product(codes, scale, wq, ws, offsets, out=i8)
        jb, j8 = guarded(n)
        moe.int8_gated(codes, scale, gq, gs, offsets, out=j8)
        db, dx = guarded(k)
        _, dw = moe.expert_product_backward(out, x, w, offsets, dx=dx)
        eb, ex = guarded(k)
        _, ew = moe.gated_product_backward(h, gu, x, gw, offsets, dx=ex)
        torch.cuda.synchronize()
        assert all(intact(b) for b in (ob, hb, gb, ib, jb, db, eb))
        assert not dw[1].any() and not ew[1].any()  # the group that ends before it begins


# ---- the same call twice, and replays --------------------------------------------------------

def calls(torch, moe, sizes, n, k, dtype, seed=0):
    """{operator: (call, its workspace, the inputs that a replay may find rewritten, offsets)}"""
    p = Case(torch, sizes, n, k, dtype, seed=seed)
    g = Case(torch, sizes, n, k, dtype, wide=2, seed=seed + 1)
    dy = p.normal(p.rows, n)
    gu = g.normal(g.rows, 2 * n)
    codes, scale = moe.quantize_rows(p.x)
    wq, ws = (a.view(*p.w.shape[:2], *a.shape[1:]) for a in moe.quantize_rows(p.w.view(-1, k)))
    gq, gs = (a.view(*g.w.shape[:2], *a.shape[1:]) for a in moe.quantize_rows(g.w.view(-1, k)))
    off = p.offsets

    def space(op):
        return sentinel(torch, max(1, moe.product_workspace(op, p.rows, n, k, len(sizes), dtype=dtype)))

    return {
        "int8_product": (lambda **kw: moe.int8_product(codes, scale, wq, ws, off, **kw), space("int8_product"), (codes, scale), off),
        "int8_gated": (lambda **kw: moe.int8_gated(codes, scale, gq, gs, off, **kw), space("int8_gated"), (codes, scale), off),
        "expert_product": (lambda **kw: moe.expert_product(p.x, p.w, off, **kw), space("expert_product"), (p.x,), off),
        "gated_product": (lambda **kw: moe.gated_product(g.x, g.w, off, save=True, **kw), space("gated_product"), (g.x,), off),
        "dx": (lambda **kw: moe.expert_product_backward(dy, p.x, p.w, off, need_dw=False, **kw)[0],
               space("expert_product_backward"), (dy, p.x), off),
        "dw": (lambda **kw: moe.expert_product_backward(dy, p.x, p.w, off, need_dx=False, **kw)[1],
               space("expert_product_backward"), (dy, p.x), off),
        "gated dx": (lambda **kw: moe.gated_product_backward(dy, gu, g.x, g.w, off, need_dw=False, **kw)[0],
                     space("gated_product_backward"), (dy, gu, g.x), off),
        "gated dw": (lambda **kw: moe.gated_product_backward(dy, gu, g.x, g.w, off, need_dx=False, **kw)[1],
                     space("gated_product_backward"), (dy, gu, g.x), off),
    }


# which operators split a contraction at these sizes (and so write raw sums to the workspace), by the
# rules of the plan; the sizes that the groups move to between replays split another number of tiles
FORWARD = ("int8_product", "int8_gated", "expert_product", "gated_product")
SPLITS = [([333, 0, 667], 1032, 8192, FORWARD), ([1000, 0, 2000], 2056, 256, ("dx", "dw")),
          ([1000, 0, 2000], 1032, 256, ("gated dx", "gated dw")), ([3000, 1, 900], 4104, 8192, FORWARD)]


@pytest.mark.parametrize("sizes,n,k,ops", SPLITS, ids=["128 forward", "128 gradients", "128 gated gradients", "256 forward"])
def test_split_calls_repeat_and_replay(torch, moe, sizes, n, k, ops):
    """Split contractions: the same bits on every call and stream, and captured into a graph whose inputs and
    offsets are rewritten between replays."""
    dtype = torch.bfloat16
    side = torch.cuda.Stream()
    made = calls(torch, moe, sizes, n, k, dtype)
    rows, groups = sum(sizes), len(sizes)
    moved = [[0, 0, 0, rows], [0, rows // 2 + 3, rows - 130, rows], [0, rows // 7, rows // 7, rows],
             [0] + [sum(sizes[:i + 1]) for i in range(groups)]]
    for op in ops:
        say(f"split {op} {sizes} {n} {k}")
        call, ws, inputs, offsets = made[op]
        first = tensors(call(workspace=ws))
        torch.cuda.synchronize()
        if op.startswith("gated d"):  # the raw sums behind (dg, du)
            assert touched(ws[rows * 4 * n:]), op
        else:
            assert touched(ws), op
        other = tensors(call(stream=side))
        with torch.cuda.stream(side):
            inside = tensors(call())
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, inside):
            assert torch.equal(a, b) and torch.equal(a, c), op
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tensors(call(workspace=ws))
        for turn, ends in enumerate(moved):
            offsets.copy_(torch.tensor(ends, dtype=torch.int32))
            for t in inputs:
                t.copy_(t.roll(1 + turn, 0))
            ws.fill_(0xFF)
            for t in out:
                t.fill_(3)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            eager = tensors(call())
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                assert torch.equal(a, b), (op, turn)
            assert not torch.equal(eager[0], first[0]) or turn == len(moved) - 1, (op, turn)
        del graph


@pytest.mark.parametrize("sizes,n,k", [([7, 0, 9, 1], 264, 208), ([70, 0, 260, 1], 1032, 144), ([900, 0, 2600, 500], 1544, 272)],
                         ids=str)
def test_replays_follow_rewritten_inputs(torch, moe, sizes, n, k):
    """Whole tiles and streaming blocks: replays take the inputs and the routing that stand there when they run,
    and leave the rows behind the last group alone."""
    rows, groups = sum(sizes), len(sizes)
    made = calls(torch, moe, sizes, n, k, torch.float16)
    turns = [[0, rows - 2, rows - 2, rows - 1, rows], [0, 0, 0, 0, rows], [0, rows // 3, rows // 2, rows // 2, rows - 3],
             [1, 1, 1, 1, 1]]
    for op, (call, ws, inputs, offsets) in made.items():
        say(f"replay {op} {sizes} {n} {k}")
        call(workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tensors(call(workspace=ws))
        whole = op.endswith("dw")  # a weight gradient has no rows of its own
        for turn, ends in enumerate(turns):
            offsets.copy_(torch.tensor(ends, dtype=torch.int32))
            for t in inputs:
                t.copy_(t.roll(1 + turn, 0))
            for t in out:
                t.fill_(3)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            eager = tensors(call())
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                assert a.shape == b.shape
                if whole:
                    assert torch.equal(a, b), (op, turn)
                else:
                    assert torch.equal(a[ends[0]:ends[-1]], b[ends[0]:ends[-1]]), (op, turn)
                    assert (a[:ends[0]] == 3).all() and (a[ends[-1]:] == 3).all(), (op, turn)
        del graph


# ---- rows of no group ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("sizes,before,after", [([5, 0, 9], 3, 6), ([0, 0, 0], 8, 8), ([40, 1, 200], 0, 100), ([], 0, 0)], ids=str)
def test_slopes_of_rows_of_no_group_are_not_computed(torch, moe, sizes, before, after, dtype):
    """The gated backward pass neither reads nor writes anything for rows before and behind the groups: the
    workspace, which starts with (dg, du) of each row, keeps what stood there."""
    n, k = 72, 64
    if not sizes:  # one group without offsets has all rows
        c = Case(torch, [17], n, k, getattr(torch, dtype), wide=2, offsets=False)
    else:
        c = Case(torch, sizes, n, k, getattr(torch, dtype), wide=2, before=before, after=after)
    m = c.member()
    dh, gu = c.normal(c.rows, n), c.normal(c.rows, 2 * n)
    ws = sentinel(torch, moe.product_workspace("gated_product_backward", c.rows, n, k, len(c.sizes), dtype=c.dtype))
    moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, workspace=ws)
    pairs = ws[: c.rows * 4 * n].view(c.rows, 4 * n)
    assert (pairs[~m] == 0xA5).all()
    assert (pairs[m] != 0xA5).any(1).all()


# ---- gradients past the range of 16 bits -----------------------------------------------------

def lifts(torch, c, d, dtype):
    """Per row, the power of two that a group's (dg, du) are divided by: 1 unless one of them leaves fp16."""
    lift = torch.ones(c.rows, 1, dtype=torch.float64, device="cuda")
    for e, b, t in c.groups():
        top = d[b:t][d[b:t].isfinite()].abs().max().item()
        if dtype == torch.float16 and top > 60000:  # (at the border either is right: the larger one bounds both)
            lift[b:t] = 2.0 ** max(0, torch.frexp(torch.tensor(top * 1.001))[1].item() - 15)
    return lift


def far_out(torch, c, n, rows, size):
    """dh and (g, u) whose product passes 65504 in some rows; small x and w keep dx and dw inside."""
    dh, gu = c.normal(c.rows, n), c.normal(c.rows, 2 * n)
    dh[rows] *= size
    gu[rows, n:] *= size
    gu[rows, :n] *= 2
    c.x.mul_(2.0 ** -8)
    c.w.mul_(2.0 ** -8)
    return dh, gu


def check_range(torch, got, ref, bound, dtype, what):
    """Within the bound where the value lies in the type's range, infinite (of its sign) where it is past it: a
    64-bit result that is itself past 65504 + 16 rounds to infinity."""
    edge = torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    past = ref.abs() - bound > edge
    assert torch.equal(got[past].double(), ref[past].sign() * float("inf")), what
    inside = ref.abs() + bound < edge
    check(torch, got[inside], ref[inside], bound[inside], what)
    return inside


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("size", [100.0, 300.0, 2000.0])
@pytest.mark.parametrize("sizes,n,k", [([70, 0, 33], 72, 136), ([333, 0, 1, 667], 1032, 256), ([700, 1500, 600], 2056, 520)], ids=str)
def test_gated_backward_past_65504(torch, moe, sizes, n, k, size, dtype, act):
    """dh u act'(g) and dh act(g) of finite fp16 values may pass the largest fp16 number; dx and dw do not.
    Those of a group are then divided by a power of two s before they are rounded, and the sums multiplied by it:
    an error of half a step, 2^-11 relative, and s times half of the smallest subnormal (2^-25)."""
    t = getattr(torch, dtype)
    c = Case(torch, sizes, n, k, t, wide=2, after=2)
    rows = torch.arange(1, sizes[0], 7, device="cuda")
    dh, gu = far_out(torch, c, n, rows, size)
    d, off = slopes64(torch, act, dh, gu, n, t)
    lift = lifts(torch, c, d, t)
    if t == torch.float16 and size >= 300:
        assert lift[0] > 1 and lift[c.ends[-2]] == 1  # only the first group
    off = off + 2.0 ** -25 * lift
    dx, dw, dx_off, dw_off = grads64(torch, c, d, off)
    got_dx, got_dw = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, activation=act)
    m = c.member()
    inside = check_range(torch, got_dx[m], dx[m], rounded(torch, dx, dx_off, t)[m], t, "dx")
    inside_dw = check_range(torch, got_dw, dw, rounded(torch, dw, dw_off, t), t, "dw")
    if size < 2000:  # nothing is infinite here
        assert inside.all() and inside_dw.all() and got_dx[m].isfinite().all() and got_dw.isfinite().all()
    none, wide = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, activation=act, need_dx=False, dw_dtype=torch.float32)
    check(torch, wide, dw, rounded(torch, dw, dw_off, torch.float32), "dw fp32")
    # the other groups' results are those of a call in which nothing is far out
    dh[rows] /= size
    gu[rows, n:] /= size
    near_dx, near_dw = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, activation=act)
    assert torch.equal(near_dx[sizes[0]:c.ends[-1]], got_dx[sizes[0]:c.ends[-1]]) and torch.equal(near_dw[1:], got_dw[1:])


def test_gated_backward_past_65504_beside_infinities(torch, moe):
    """An infinite dh is not a large one: its row and its columns of dw are not finite, the others are right."""
    t, n, k = torch.float16, 72, 136
    c = Case(torch, [40, 30], n, k, t, wide=2)
    dh, gu = far_out(torch, c, n, torch.tensor([3, 50], device="cuda"), 300.0)
    dh[5, 7] = float("inf")
    dh[51, 2] = float("nan")
    dx, dw = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets)
    rest = torch.ones(70, dtype=torch.bool, device="cuda")
    rest[[5, 51]] = False
    assert dx[rest].isfinite().all() and not dx[5].isfinite().any() and dx[51].isnan().all()
    cols = torch.ones(2, 2 * n, dtype=torch.bool, device="cuda")
    cols[0, [7, n + 7]] = False
    cols[1, [2, n + 2]] = False
    assert dw[cols].isfinite().all() and not dw[~cols].isfinite().any()
    clean = dh.clone()
    clean[5, 7], clean[51, 2] = 0, 0
    d, off = slopes64(torch, "silu", clean, gu, n, t)
    off = off + 2.0 ** -25 * lifts(torch, c, d, t)
    rx, rw, rx_off, rw_off = grads64(torch, c, d, off)
    check(torch, dx[rest], rx[rest], rounded(torch, rx, rx_off, t)[rest], "dx")
    check(torch, dw[cols], rw[cols], rounded(torch, rw, rw_off, t)[cols], "dw")


def test_gated_backward_past_65504_replays(torch, moe):
    """A captured call scales where the inputs of a replay ask for it, and not on the next."""
    t, n, k = torch.float16, 264, 136
    c = Case(torch, [40, 300], n, k, t, wide=2)
    near = (c.normal(340, n), c.normal(340, 2 * n))
    c.x.mul_(2.0 ** -8)
    c.w.mul_(2.0 ** -8)
    dh, gu = (a.clone() for a in near)
    ws = sentinel(torch, moe.product_workspace("gated_product_backward", 340, n, k, 2, dtype=t))
    moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets, workspace=ws)
    for rows in ([], [5], [100, 7], [], [200]):
        dh.copy_(near[0])
        gu.copy_(near[1])
        dh[rows] *= 300.0
        gu[rows, n:] *= 300.0
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = moe.gated_product_backward(dh, gu, c.x, c.w, c.offsets)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert a.isfinite().all() and torch.equal(a, b), rows
    del graph


# ---- gradients of one side only ------------------------------------------------------------

@pytest.mark.parametrize("sizes", [[40, 0, 17], [57]], ids=str)
def test_backward_without_the_other_operand(torch, moe, sizes):
    """dx needs no x, dw needs no w: the results are those of the call that has both."""
    n, k, bf16 = 72, 136, torch.bfloat16
    for wide in (1, 2):
        c = Case(torch, sizes, n, k, bf16, wide=wide, offsets=len(sizes) > 1)
        w = c.w if len(sizes) > 1 else c.w[0]
        dy, gu = c.normal(c.rows, n), c.normal(c.rows, 2 * n)

        def call(x, w, **kw):
            if wide == 2:
                return moe.gated_product_backward(dy, gu, x, w, c.offsets, **kw)
            return moe.expert_product_backward(dy, x, w, c.offsets, **kw)

        dx, dw = call(c.x, w)
        only, none = call(None, w, need_dw=False)
        assert none is None and torch.equal(only, dx)
        none, only = call(c.x, None, need_dx=False)
        assert none is None and only.shape == dw.shape and torch.equal(only, dw)
        given = torch.empty(dw.shape, dtype=torch.float32, device="cuda")
        _, only = call(c.x, None, need_dx=False, dw=given)
        assert only is given and torch.equal(only.to(bf16), dw)
        with pytest.raises(ValueError, match="x is needed"):
            call(None, w)
        with pytest.raises(ValueError, match="w is needed"):
            call(c.x, None)
        with pytest.raises(ValueError, match="dw must be"):
            call(c.x, None, need_dx=False, dw=given[..., :8].contiguous())


# ---- autograd ---------------------------------------------------------------------------------

def test_tensors_that_autograd_tracks_are_refused(torch, moe):
    """No call records anything for autograd, so one that autograd expects a gradient from is refused: a result cut
    off without a word would train nothing."""
    bf16 = torch.bfloat16
    x, w = torch.randn(4, 64, device="cuda").to(bf16), torch.randn(1, 48, 64, device="cuda").to(bf16)
    dy, gu = torch.randn(4, 24, device="cuda").to(bf16), torch.randn(4, 48, device="cuda").to(bf16)
    codes, scale = moe.quantize_rows(x)
    wq, ws = torch.ones(1, 48, 64, dtype=torch.int8, device="cuda"), torch.ones(1, 48, device="cuda")
    every = [(moe.quantize_rows, (x,)), (moe.expert_product, (x, w)), (moe.gated_product, (x, w)),
             (moe.int8_product, (codes, scale, wq, ws)), (moe.int8_gated, (codes, scale, wq, ws)),
             (moe.gated_product_backward, (dy, gu, x, w)), (moe.expert_product_backward, (gu, x, w))]
    for fn, args in every:
        ref = tensors(fn(*args))
        for i, a in enumerate(args):
            if not a.is_floating_point():
                continue
            leaf = list(args)
            leaf[i] = a.detach().clone().requires_grad_()
            with pytest.raises(ValueError, match="autograd"):
                fn(*leaf)
            with torch.no_grad():
                for b, c in zip(tensors(fn(*leaf)), ref):
                    assert torch.equal(b, c) and not b.requires_grad


# ---- subnormal operands and results -------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", [([9, 0, 3], 72, 136), ([700, 0, 900], 1544, 144), ([5000, 1, 333], 1032, 144)], ids=str)
def test_subnormal_values(torch, moe, sizes, n, k, dtype):
    """Operands below the type's normal range count in full, and results there are rounded to its subnormals."""
    t = getattr(torch, dtype)
    tiny = torch.finfo(t).smallest_normal
    half_subnormal = tiny * torch.finfo(t).eps / 2
    c = Case(torch, sizes, n, k, t)
    # bf16 shares fp32's exponents: there the other operand lifts the results to about 2^-122, and one below the
    # normal range (2^-126) may be flushed
    c.x = (c.x.double() * tiny / 4).to(t)
    c.w = (c.w.double() * (1 if t == torch.float16 else 64)).to(t)
    y, before = c.forward()
    bound = before + half_step(torch, t) * (y.abs() + before) + half_subnormal + 2.0 ** -126 * (t == torch.bfloat16)
    check(torch, moe.expert_product(c.x, c.w, c.offsets), y, bound, "y")
    dy = (c.normal(c.rows, n).double() * tiny / 8).to(t)
    dx, _, dx_off, _ = grads64(torch, c, dy.double(), torch.zeros(c.rows, n, dtype=torch.float64, device="cuda"))
    bound = dx_off + half_step(torch, t) * (dx.abs() + dx_off) + half_subnormal + 2.0 ** -126 * (t == torch.bfloat16)
    check(torch, moe.expert_product_backward(dy, c.x, c.w, c.offsets, need_dw=False)[0], dx, bound, "dx")
