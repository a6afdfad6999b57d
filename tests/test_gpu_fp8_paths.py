"""The products in 8-bit floating point on the GPU beyond their plain calls:
rows of no group, strides, infinities and NaN, streams, replays, workspaces,
offsets out of order, long matrices, gradients against differences, and the
training step that they make up with the products in 16 bits and AdamW."""

import pytest

from gpu_util import require_gpu, say
from test_gpu_fp8 import Case, blocks, blocks64, rounded, slopes64, spread, tiles64
from test_gpu_products import E, act64, check, gated64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


def bits(t):
    """The same memory as whole numbers (8-bit floats have few operations)."""
    import torch
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


SIZES = [([5, 0, 9], 80, 208), ([100, 0, 150, 3], 272, 208), ([1500, 0, 700, 3], 528, 4112), ([2000, 1500], 2560, 80)]


@pytest.mark.parametrize("sizes,n,k", SIZES, ids=str)
def test_rows_of_no_group_and_strides(torch, moe, sizes, n, k):
    """Rows before and behind the groups hold NaN and are neither read nor written, nor is the space between rows."""
    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn

    def rows_of(c):
        """The codes in wider rows, and the scales in longer blocks, all else NaN."""
        m = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
        m[c.ends[0]:c.ends[-1]] = True
        buf = torch.full((c.rows, c.width + 48), 0x7F, dtype=torch.uint8, device="cuda")
        buf[m, :c.width] = c.codes.view(torch.uint8)[m]
        scale = torch.full((blocks(c.width), c.rows + 5), float("nan"), device="cuda")
        scale[:, :c.rows][:, m] = c.scale[:, m]
        return m, buf.view(e4m3)[:, :c.width], scale[:, :c.rows]

    def buffers(rows, width):
        buf = torch.full((rows, width + 8), 7.0, dtype=bf16, device="cuda")
        return buf, buf[:, :width]

    def untouched(buf, m, width):
        assert (buf[~m] == 7.0).all() and (buf[:, width:] == 7.0).all()

    c = Case(torch, sizes, n, k, before=3, after=6)
    m, codes, scale = rows_of(c)
    y, s = c.product()
    buf, out = buffers(c.rows, n)
    assert moe.fp8_product(codes, scale, c.w, c.w_scale, c.offsets, out=out) is out
    untouched(buf, m, n)
    check(torch, out[m], y[m], rounded(torch, y, s, bf16)[m], "y")

    c = Case(torch, sizes, n, k, gated=True, before=3, after=6)
    m, codes, scale = rows_of(c)
    y, s = c.product()
    h, before = gated64(torch, "silu", y[:, :n], y[:, n:], s[:, :n], s[:, n:])
    hb, hv = buffers(c.rows, n)
    kb, kv = buffers(c.rows, 2 * n)
    moe.fp8_gated(codes, scale, c.w, c.w_scale, c.offsets, out=hv, gate_up=kv)
    untouched(hb, m, n)
    untouched(kb, m, 2 * n)
    check(torch, hv[m], h[m], rounded(torch, h, before, bf16)[m], "h")
    check(torch, kv[m], y[m], rounded(torch, y, s, bf16)[m], "gate_up")

    b = Case(torch, sizes, n, k, backward=True, before=3, after=6)
    _, codes, scale = rows_of(b)
    dx, s = b.product(backward=True)
    buf, got = buffers(b.rows, k)
    moe.fp8_product_backward(codes, scale, b.w, b.w_scale, b.offsets, dx=got)
    untouched(buf, m, k)
    check(torch, got[m], dx[m], rounded(torch, dx, s, bf16)[m], "dx")

    dh = torch.full((c.rows, n + 16), float("nan"), dtype=bf16, device="cuda")
    dh[m, :n] = torch.randn(int(m.sum()), n, device="cuda").to(bf16)
    kv[~m] = float("nan")
    clean = moe.fp8_gated_backward(dh[:, :n].nan_to_num(0.0), kv.nan_to_num(0.0).contiguous(), c.w, c.w_scale, c.offsets)
    buf, got = buffers(c.rows, k)
    sb, sv = buffers(c.rows, 2 * n)
    moe.fp8_gated_backward(dh[:, :n], kv, c.w, c.w_scale, c.offsets, dx=got, slopes=sv)
    untouched(buf, m, k)
    untouched(sb, m, 2 * n)
    assert torch.equal(got[m], clean[0][m]) and torch.equal(sv[m], clean[1][m])


@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_given_buffers(torch, moe, tiles):
    x = torch.randn(80, 272, device="cuda").to(torch.bfloat16)
    ref = moe.quantize_blocks(x, tiles=tiles)
    if tiles:
        codes, scale = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    else:
        codes = torch.zeros(80, 272 + 32, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, 16:-16]
        scale = torch.full((3, 100), 5.0, device="cuda")
        wide = torch.full((80, 272 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 8:280] = x
        x = wide[:, 8:280]
        scale, whole = scale[:, 7:87], scale
    moe.quantize_blocks(x, tiles=tiles, codes=codes, scale=scale)
    assert torch.equal(bits(codes.contiguous()), bits(ref[0])) and torch.equal(scale, ref[1])
    if not tiles:
        assert (whole[:, :7] == 5.0).all() and (whole[:, 87:] == 5.0).all()


@pytest.mark.parametrize("rows,n,k", [(5, 80, 400), (300, 272, 400), (700, 1552, 8208), (3000, 4112, 400)], ids=str)
def test_nan_stays_in_its_row_and_column(torch, moe, rows, n, k):
    """A scale or a code that is NaN makes NaN of the results that it takes part in, and of no others."""
    sizes = [rows, rows // 2]
    for gated in (False, True):
        c = Case(torch, sizes, n, k, gated=gated)
        c.scale[0, 1] = float("nan")
        c.scale[blocks(k) - 1, rows - 1] = float("nan")
        c.codes.view(torch.uint8)[3, 129] = 0x7F
        call = (lambda: moe.fp8_gated(c.codes, c.scale, c.w, c.w_scale, c.offsets)) if gated else (
            lambda: moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, c.offsets))
        y = call()
        bad = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
        bad[[1, 3, rows - 1]] = True
        assert y[bad].isnan().all() and y[~bad].isfinite().all()
    c = Case(torch, sizes, n, k)
    c.w_scale[1, 0, 0] = float("nan")            # columns 0 .. 127 of the second group
    c.w.view(torch.uint8)[0, n - 1, 3] = 0x7F   # the last column of the first
    y = moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, c.offsets)
    hit = torch.zeros(c.rows, n, dtype=torch.bool, device="cuda")
    hit[rows:, :128] = True
    hit[:rows, n - 1] = True
    assert y[hit].isnan().all() and y[~hit].isfinite().all()
    b = Case(torch, sizes, n, k, backward=True)
    b.w_scale[1, 0, 1] = float("nan")            # columns 128 .. 255 of dx, of the second group
    b.w.view(torch.uint8)[0, n - 1, 3] = 0x7F
    dx = moe.fp8_product_backward(b.codes, b.scale, b.w, b.w_scale, b.offsets)
    hit = torch.zeros(b.rows, k, dtype=torch.bool, device="cuda")
    hit[rows:, 128:256] = True
    hit[:rows, 3] = True
    assert dx[hit].isnan().all() and dx[~hit].isfinite().all()
    g = Case(torch, sizes, n, k, gated=True)
    dh = torch.randn(g.rows, n, device="cuda").to(torch.bfloat16)
    gu = torch.randn(g.rows, 2 * n, device="cuda").to(torch.bfloat16)
    dh[1, 0] = float("nan")
    dh[2, n - 1] = float("inf")
    gu[3, n] = float("-inf")
    dx, slopes = moe.fp8_gated_backward(dh, gu, g.w, g.w_scale, g.offsets)
    rest = torch.ones(g.rows, dtype=torch.bool, device="cuda")
    rest[1:4] = False
    assert dx[1:4].isnan().all() and dx[rest].isfinite().all() and slopes[rest].isfinite().all()
    # up's last and gate's first rows meet in a stage of the contraction: NaN codes in one reach no row that they
    # do not belong to, and every row of their group that they do
    g.w.view(torch.uint8)[0, 1, 0, 5] = 0x7F
    dx, _ = moe.fp8_gated_backward(dh, gu, g.w, g.w_scale, g.offsets)
    keep = rest[:, None] & (torch.arange(k, device="cuda") != 5)
    keep[rows:] = rest[rows:, None]
    assert dx[:rows, 5].isnan().all() and dx[keep].isfinite().all()


def test_fp16_slopes_past_65504(torch, moe):
    """A slope that fp16 cannot hold is infinite in the slopes and finite on its way through the codes."""
    sizes, n, k = [40, 50], 144, 272
    c = Case(torch, sizes, n, k, gated=True)
    c.w_scale *= 1e-4
    t = torch.float16
    dh = torch.randn(90, n, generator=c.gen, device="cuda").to(t)
    gu = torch.randn(90, 2 * n, generator=c.gen, device="cuda").to(t)
    dh[7, 3], gu[7, 3], gu[7, n + 3] = 3000.0, 2.0, 500.0
    dx, slopes = moe.fp8_gated_backward(dh, gu, c.w, c.w_scale, c.offsets)
    assert slopes[7, 3].isinf() and dx.isfinite().all()
    dg, du, dg_off, du_off = slopes64(torch, "silu", dh, gu, n)
    # the codes are within half a step of the slopes: 2^-4 of themselves, 2^-10 of their block's scale
    x = torch.cat([dg, du], 1)
    step = torch.cat([spread(blocks64(torch, d)[1].t(), n) for d in (dg, du)], 1)
    off = x.abs() * 2.0 ** -4 * (1 + 1e-3) + step * 2.0 ** -10 + torch.cat([dg_off, du_off], 1)
    ref, _ = c.product(x, backward=True)
    _, s = c.product(x.abs() + off, backward=True)
    m = torch.zeros_like(ref)
    for e, b, u in c.groups():
        m[b:u] = off[b:u] @ c.w64(e).abs()
    check(torch, dx, ref, rounded(torch, ref, m + s, t), "dx")


def every_call(torch, moe, sizes, n, k):
    p, g = Case(torch, sizes, n, k), Case(torch, sizes, n, k, gated=True, seed=1)
    b = Case(torch, sizes, n, k, backward=True, seed=2)
    x = torch.randn(p.rows, k, generator=p.gen, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, n, k, generator=p.gen, device="cuda").to(torch.float16)
    dh = torch.randn(p.rows, n, generator=p.gen, device="cuda").to(torch.bfloat16)
    gu = torch.randn(p.rows, 2 * n, generator=p.gen, device="cuda").to(torch.bfloat16)
    return [
        ("rows", None, (x,), lambda **kw: moe.quantize_blocks(x, **kw)),
        ("tiles", None, (w,), lambda **kw: moe.quantize_blocks(w, tiles=True, **kw)),
        ("fp8_product", p, (p.codes, p.scale), lambda **kw: moe.fp8_product(p.codes, p.scale, p.w, p.w_scale, p.offsets, **kw)),
        ("fp8_gated", g, (g.codes, g.scale),
         lambda **kw: moe.fp8_gated(g.codes, g.scale, g.w, g.w_scale, g.offsets, save=True, **kw)),
        ("fp8_product_backward", b, (b.codes, b.scale),
         lambda **kw: moe.fp8_product_backward(b.codes, b.scale, b.w, b.w_scale, b.offsets, **kw)),
        ("fp8_gated_backward", g, (dh, gu),
         lambda **kw: moe.fp8_gated_backward(dh, gu, g.w, g.w_scale, g.offsets, **kw)),
    ]


def tensors(result):
    return list(result) if isinstance(result, tuple) else [result]


# few rows, 128-wide tiles split, 256-wide ones with the last round's remainder split
RUNS = [([3, 0, 4], 144, 4112), ([300, 0, 500], 1040, 4112), ([3000, 1, 900], 4112, 4112)]


@pytest.mark.parametrize("sizes,n,k", RUNS, ids=str)
def test_same_bits_on_any_stream(torch, moe, sizes, n, k):
    side = torch.cuda.Stream()
    for name, _, _, call in every_call(torch, moe, sizes, n, k):
        first = tensors(call())
        torch.cuda.synchronize()
        other = tensors(call(stream=side))
        with torch.cuda.stream(side):
            inside = tensors(call())
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, inside):
            assert torch.equal(bits(a), bits(b)) and torch.equal(bits(a), bits(c)), name


@pytest.mark.parametrize("sizes,n,k", RUNS, ids=str)
def test_captured_calls_replay(torch, moe, sizes, n, k):
    """Each call captured over a workspace that holds anything; replays follow rewritten inputs and offsets, with eager
    work between them."""
    for name, case, inputs, call in every_call(torch, moe, sizes, n, k):
        kw = {}
        if case is not None:
            need = moe.fp8_workspace(name, case.rows, n, k, len(sizes))
            kw["workspace"] = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tensors(call(**kw))
        for turn in range(3):
            for t in out:
                bits(t).zero_()
            if turn and case is not None:  # other rows to the groups, and other rows
                ends = case.offsets.clone()
                ends[1:-1] = case.rows * turn // 4
                case.offsets.copy_(ends)
                if turn == 2:
                    kw["workspace"].fill_(0x7F)
            for t in inputs:
                bits(t).copy_(bits(t).roll(turn, -1))
            graph.replay()
            eager = tensors(call())
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                assert torch.equal(bits(a), bits(b)), (name, turn)
        del graph


def test_two_graphs_share_a_workspace(torch, moe):
    cases = [Case(torch, [2000], 1024, 8192), Case(torch, [1900], 1040, 4112, seed=1)]
    needs = [moe.fp8_workspace("fp8_product", c.rows, c.n, c.k) for c in cases]
    assert min(needs) > 0
    ws = torch.empty(max(needs), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(c.rows, c.n, dtype=torch.bfloat16, device="cuda") for c in cases]
    refs = [moe.fp8_product(c.codes, c.scale, c.w, c.w_scale) for c in cases]
    torch.cuda.synchronize()
    graphs = []
    for c, out in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, out=out, workspace=ws)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0)):
        for o in outs:
            o.zero_()
        ws.fill_(0xFF)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])


def test_one_matrix_and_refusals(torch, moe):
    c = Case(torch, [40], 144, 272)
    ref = moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, c.offsets)
    assert torch.equal(moe.fp8_product(c.codes, c.scale, c.w[0], c.w_scale[0]), ref)
    g = Case(torch, [40], 144, 272, gated=True)
    ref = moe.fp8_gated(g.codes, g.scale, g.w, g.w_scale, g.offsets)
    assert torch.equal(moe.fp8_gated(g.codes, g.scale, g.w[0], g.w_scale[0]), ref)
    one = Case(torch, [1], 144, 272)
    ref = moe.fp8_product(one.codes, one.scale, one.w, one.w_scale)
    lying = one.scale.t().contiguous().t()  # a single row's scales, in any layout
    assert torch.equal(moe.fp8_product(one.codes, lying, one.w, one.w_scale), ref)
    args = dict(codes=c.codes, scale=c.scale, w=c.w, w_scale=c.w_scale, offsets=c.offsets)

    def refused(error, match, **over):
        with pytest.raises(error, match=match):
            moe.fp8_product(**{**args, **over})

    refused(ValueError, "codes must be", codes=c.codes.view(torch.int8))
    refused(ValueError, "codes must be", codes=c.codes[:, :256])
    refused(ValueError, "scale must be", scale=c.scale.t().contiguous())
    refused(ValueError, "scale must be", scale=c.scale.double())
    refused(ValueError, "scale is on", scale=c.scale.cpu())
    refused(ValueError, "contiguous", scale=c.scale.t().contiguous().t())
    refused(ValueError, "w_scale must be", w_scale=c.w_scale[:, :1])
    refused(ValueError, "contiguous", w=c.w.transpose(1, 2).contiguous().transpose(1, 2))
    refused(ValueError, "offsets must be", offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    refused(moe.MoeError, "type", dtype=torch.float32)
    refused(ValueError, "unsupported dtype", dtype=torch.float64)
    refused(moe.MoeError, "stride", codes=c.codes[:1].expand(40, -1))   # rows on top of each other
    refused(moe.MoeError, "scale", scale=c.scale[:1].expand(3, -1))
    with pytest.raises(moe.MoeError, match="aligned|stride"):
        moe.quantize_blocks(torch.zeros(8, 100, dtype=torch.bfloat16, device="cuda")[:, 4:84])
    with pytest.raises(ValueError, match="contiguous"):
        moe.quantize_blocks(torch.zeros(64, 160, dtype=torch.bfloat16, device="cuda")[:, :64], tiles=True)
    with pytest.raises(moe.MoeError):
        moe.quantize_blocks(torch.zeros(64, 64, device="cuda"))
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="autograd"):
        moe.quantize_blocks(x)
    with torch.no_grad():
        moe.quantize_blocks(x)
    with pytest.raises(ValueError, match="gate_up must be"):
        moe.fp8_gated_backward(torch.zeros(40, 144, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(40, 288, dtype=torch.float16, device="cuda"), g.w, g.w_scale)
    torch.cuda.synchronize()


def test_offsets_out_of_order_or_range(torch, moe):
    """Groups that overlap, end before they begin or leave the rows: every call stays inside its matrices."""
    n, k = 1040, 144
    for s in (1, 10, 40):  # few rows, 128- and 256-wide tiles
        r = 200 * s
        offsets = torch.tensor([-5, 100 * s, 60 * s, 1 << 30], dtype=torch.int32, device="cuda")
        c = Case(torch, [r, 0, 0], n, k)
        g = Case(torch, [r, 0, 0], n, k, gated=True)
        b = Case(torch, [r, 0, 0], n, k, backward=True)

        def guarded(width):
            buf = torch.full((r + 20, width), 7.0, dtype=torch.bfloat16, device="cuda")
            return buf, buf[10:-10]

        (ob, out), (hb, h), (gb, gu), (db, dx), (eb, ex), (sb, sl) = (
            guarded(x) for x in (n, n, 2 * n, k, k, 2 * n))
        moe.fp8_product(c.codes, c.scale, c.w, c.w_scale, offsets, out=out)
        moe.fp8_gated(g.codes, g.scale, g.w, g.w_scale, offsets, out=h, gate_up=gu)
        moe.fp8_product_backward(b.codes, b.scale, b.w, b.w_scale, offsets, dx=dx)
        moe.fp8_gated_backward(h, gu, g.w, g.w_scale, offsets, dx=ex, slopes=sl)
        torch.cuda.synchronize()
        for buf in (ob, hb, gb, db, eb, sb):
            assert (buf[:10] == 7.0).all() and (buf[-10:] == 7.0).all()


def test_no_rows(torch, moe):
    """Calls without rows, and with only empty groups: nothing is written."""
    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn
    w, ws = moe.quantize_blocks(torch.ones(3, 48, 64, dtype=bf16, device="cuda"), tiles=True)
    gw, gs = moe.quantize_blocks(torch.ones(3, 2, 48, 64, dtype=bf16, device="cuda"), tiles=True)
    for rows in (0, 5, 300):
        off = torch.full((4,), rows // 2, dtype=torch.int32, device="cuda")
        codes, scale = moe.quantize_blocks(torch.ones(rows, 64, dtype=bf16, device="cuda"))
        assert codes.shape == (rows, 64) and scale.shape == (1, rows) and codes.dtype == e4m3
        dcodes, dscale = moe.quantize_blocks(torch.ones(rows, 48, dtype=bf16, device="cuda"))

        def full(width):
            return torch.full((rows, width), 3.0, dtype=bf16, device="cuda")

        outs = [moe.fp8_product(codes, scale, w, ws, off, out=full(48)),
                *moe.fp8_gated(codes, scale, gw, gs, off, out=full(48), gate_up=full(96)),
                moe.fp8_product_backward(dcodes, dscale, w, ws, off, dx=full(64)),
                *moe.fp8_gated_backward(full(48), full(96), gw, gs, off, dx=full(64), slopes=full(96))]
        assert all((o == 3.0).all() for o in outs)
    assert moe.quantize_blocks(torch.zeros(0, 2, 48, 64, dtype=bf16, device="cuda"), tiles=True)[1].shape == (0, 2, 1, 1)


def test_past_32_bits(torch, moe):
    """Row matrices and weights of more than 4 GiB: the last rows and the last group."""
    bf16 = torch.bfloat16
    rows, k, n = 1_200_000, 4096, 16
    x = torch.zeros(rows, k, dtype=bf16, device="cuda")
    tail = torch.randn(300, k, device="cuda").to(bf16)
    x[-300:] = tail
    codes, scale = moe.quantize_blocks(x)
    del x
    ref_codes, ref_scale = moe.quantize_blocks(tail)
    assert torch.equal(bits(codes[-300:].contiguous()), bits(ref_codes)) and torch.equal(scale[:, -300:], ref_scale)
    assert not codes.view(torch.uint8)[:-300].any() and not scale[:, :-300].any()
    w, w_scale = moe.quantize_blocks((torch.randn(2, n, k, device="cuda") / 64).to(bf16), tiles=True)
    off = torch.tensor([0, rows - 300, rows], dtype=torch.int32, device="cuda")
    y = moe.fp8_product(codes, scale, w, w_scale, off)
    alone = moe.fp8_product(ref_codes, ref_scale, w[1], w_scale[1])
    # other tiles of the rows, so the waves' sums may meet in another order
    s = ((ref_codes.double() * spread(ref_scale.t(), k)).abs() @ (w[1].double() * spread(w_scale[1], k)).abs().t().contiguous())
    assert ((y[-300:].double() - alone.double()).abs() <= 2.0 ** -8 * alone.double().abs() * 1.01 + 100 * E * s).all()
    assert not y[:-300].any()
    dx = moe.fp8_product_backward(*moe.quantize_blocks(y), w, w_scale, off)
    assert dx[-300:].any() and not dx[:-300].any()
    del codes, scale, y, dx
    groups, n, k = 70, 8192, 8192  # 4.7 GB of weights in codes
    w = torch.zeros(groups, n, k, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    last, last_scale = moe.quantize_blocks((torch.randn(n, k, device="cuda") / 90).to(bf16), tiles=True)
    w[-1] = last
    w_scale = torch.ones(groups, blocks(n), blocks(k), device="cuda")
    w_scale[-1] = last_scale
    for count in (3, 100, 2000):
        codes, scale = moe.quantize_blocks(torch.randn(count + groups - 1, k, device="cuda").to(bf16))
        off = torch.tensor(list(range(groups)) + [count + groups - 1], dtype=torch.int32, device="cuda")
        x64 = codes[-count:].double() * spread(scale.t()[-count:], k)
        w64 = last.double() * spread(last_scale, k).repeat_interleave(128, 0)
        ref = x64 @ w64.t().contiguous()
        # a product is cut off at 2^-13 of the largest: 2^-6 of the blocks' largest values' products
        cut = 2.0 ** -6 * (scale.t()[-count:].double() * 448) @ (last_scale.double() * 448).t().contiguous().repeat_interleave(128, 1)
        bound = cut + 400 * E * (x64.abs() @ w64.abs().t().contiguous())
        y = moe.fp8_product(codes, scale, w, w_scale, off)
        check(torch, y[-count:], ref, rounded(torch, ref, bound, bf16), "last group")
        assert not y[:-count].any()
        dx = moe.fp8_product_backward(codes, scale, w, w_scale, off)
        ref = x64 @ w64
        cut = 2.0 ** -6 * (scale.t()[-count:].double() * 448) @ (last_scale.double() * 448).repeat_interleave(128, 1)
        check(torch, dx[-count:], ref, rounded(torch, ref, cut + 400 * E * (x64.abs() @ w64.abs()), bf16), "last group dx")
        assert not dx[:-count].any()


# ---- gradients against differences --------------------------------------------------------

def test_rows_past_a_grid(torch, moe):
    """More rows than one dimension of the grid takes: 2^19 of quantize_blocks, 2^18 of the slopes.  Rows do not
    depend on each other, so parts of them give the same bits."""
    say("700001 rows")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(700001, 528, generator=gen, device="cuda").bfloat16()
    codes, scale = moe.quantize_blocks(x)
    for at in range(0, x.shape[0], 200000):
        part, ps = moe.quantize_blocks(x[at:at + 200000])
        assert torch.equal(bits(part), bits(codes[at:at + 200000]))
        assert torch.equal(ps, scale[:, at:at + 200000])
    del x, codes, scale
    rows, n, k = 600001, 144, 16
    dh = torch.randn(rows, n, generator=gen, device="cuda").bfloat16()
    gate_up = torch.randn(rows, 2 * n, generator=gen, device="cuda").bfloat16()
    w, ws = moe.quantize_blocks(torch.randn(1, 2, n, k, generator=gen, device="cuda").bfloat16(), tiles=True)
    dx, slopes = moe.fp8_gated_backward(dh, gate_up, w, ws)
    for at in range(0, rows, 200000):
        pdx, ps = moe.fp8_gated_backward(dh[at:at + 200000], gate_up[at:at + 200000], w, ws)
        assert torch.equal(pdx, dx[at:at + 200000])
        assert torch.equal(ps, slopes[at:at + 200000])


def test_product_gradient_against_differences(torch, moe):
    """Small whole codes and scales that are powers of two: every sum is exact in fp16, so that dx equals the
    differences of <dy, y> along each value of x, bit for bit."""
    sizes, n, k, t = [9, 0, 23], 48, 144, torch.float16
    gen = torch.Generator(device="cuda").manual_seed(3)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").float()

    rows = sum(sizes)
    off = torch.tensor([0, 9, 9, 32], dtype=torch.int32, device="cuda")
    w = whole(3, n, k).to(torch.float8_e4m3fn)
    w_scale = torch.exp2(torch.randint(-1, 1, (3, blocks(n), blocks(k)), generator=gen, device="cuda").float())
    x, dy = whole(rows, k), whole(rows, n)
    one = torch.ones(blocks(k), rows, device="cuda")
    dx = moe.fp8_product_backward(dy.to(torch.float8_e4m3fn), torch.ones(blocks(n), rows, device="cuda"), w, w_scale, off,
                                  dtype=t)
    for at in (0, 1, 77, 127, 128, 143):
        up, down = x.clone(), x.clone()
        up[:, at] += 1
        down[:, at] -= 1
        y = [moe.fp8_product(v.to(torch.float8_e4m3fn), one, w, w_scale, off, dtype=t).double() for v in (up, down)]
        slope = ((y[0] - y[1]) * dy.double()).sum(1) / 2
        assert torch.equal(dx[:, at].double(), slope)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_slopes_against_differences(torch, moe, act):
    """(dg, du) against central differences of L = sum dh act(g) u in 64 bits, and dx against them through w."""
    sizes, n, k = [30, 0, 41], 144, 80
    c = Case(torch, sizes, n, k, gated=True)
    dh = torch.randn(c.rows, n, generator=c.gen, device="cuda").half()
    gu = torch.randn(c.rows, 2 * n, generator=c.gen, device="cuda").half()
    dx, slopes = moe.fp8_gated_backward(dh, gu, c.w, c.w_scale, c.offsets, activation=act)
    g, u, d = gu[:, :n].double(), gu[:, n:].double(), dh.double()
    eps = 1e-4

    def loss(g, u):
        return d * act64(torch, act, g)[0] * u

    dg = (loss(g + eps, u) - loss(g - eps, u)) / (2 * eps)
    du = (loss(g, u + eps) - loss(g, u - eps)) / (2 * eps)
    ref = torch.cat([dg, du], 1)
    # the difference's own error: eps^2 / 6 of a third derivative below 2 |dh u|, and 64-bit rounding over eps
    own = torch.cat([(d * u).abs(), d.abs() * 4], 1) * eps * eps + 1e-11
    _, _, dg_off, du_off = slopes64(torch, act, dh, gu, n)
    off = own + torch.cat([dg_off, du_off], 1)
    check(torch, slopes, ref, rounded(torch, ref, off, torch.float16), "slopes")
    # half a step of the codes beside it: 2^-4 of a slope, 2^-10 of its block's scale
    step = torch.cat([spread(blocks64(torch, s)[1].t(), n) for s in (dg, du)], 1)
    moved = off + ref.abs() * 2.0 ** -4 * (1 + 1e-3) + step * 2.0 ** -10
    want, _ = c.product(ref, backward=True)
    _, s = c.product(ref.abs() + moved, backward=True)
    m = torch.zeros_like(want)
    for e, b, t in c.groups():
        m[b:t] = moved[b:t] @ c.w64(e).abs()
    check(torch, dx, want, rounded(torch, want, m + s, torch.float16), "dx")


# ---- together -------------------------------------------------------------------------------

def test_a_training_step_of_the_experts(torch, moe):
    """Weights into codes, the block forward and backward in codes, the weights' gradients in 16 bits, AdamW, and the
    new weights into codes: each step equals its formula on what the one before it left."""
    sizes, d, f = [50, 0, 131, 75], 272, 400
    bf16 = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows, e = sum(sizes), len(sizes)
    off = torch.tensor([0, 50, 50, 181, 256], dtype=torch.int32, device="cuda")

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    master = [normal(e, 2, f, d, std=d ** -0.5), normal(e, d, f, std=f ** -0.5)]
    params = [w.to(bf16) for w in master]
    states = moe.adamw_states(params, bits=8)
    x, dy = normal(rows, d).to(bf16), normal(rows, d).to(bf16)
    with torch.no_grad():
        for step in (1, 2):
            (wg, sg), (wd, sd) = (moe.quantize_blocks(p, tiles=True) for p in params)
            ref, s = tiles64(torch, params[0])
            assert torch.equal(wg.double(), ref)
            xq, xs = moe.quantize_blocks(x)
            h, gu = moe.fp8_gated(xq, xs, wg, sg, off, save=True)
            hq, hs = moe.quantize_blocks(h)
            y = moe.fp8_product(hq, hs, wd, sd, off)
            dq, ds = moe.quantize_blocks(dy)
            dh = moe.fp8_product_backward(dq, ds, wd, sd, off)
            dx, slopes = moe.fp8_gated_backward(dh, gu, wg, sg, off)
            _, dwd = moe.expert_product_backward(dy, h, None, off, need_dx=False)
            _, dwg = moe.expert_product_backward(slopes, x, None, off, need_dx=False)
            # the same block in 64 bits on the codes' values: every stage is within its own bound of the formula,
            # so the whole is near it: 2^-4 a code, and three codes in a row
            x64, y64, dx64 = xq.double() * spread(xs.t(), d), torch.zeros(rows, d).double().cuda(), torch.zeros(rows, d).double().cuda()
            begin = 0
            for g, size in enumerate(sizes):
                t = slice(begin, begin + size)
                begin += size
                w1 = (wg[g].double() * spread(sg[g], d).repeat_interleave(128, 1)[:, :f])
                w2 = wd[g].double() * spread(sd[g], f).repeat_interleave(128, 0)[:d]
                gate, up = x64[t] @ w1[0].t().contiguous(), x64[t] @ w1[1].t().contiguous()
                a, slope, _, _ = act64(torch, "silu", gate)
                y64[t] = (a * up) @ w2.t().contiguous()
                dh64 = dy[t].double() @ w2
                dx64[t] = (dh64 * up * slope) @ w1[0] + (dh64 * a) @ w1[1]
            for got, want in ((y, y64), (dx, dx64)):
                assert (got.double() - want).norm() <= 3 * 2.0 ** -4 * want.norm()
            before = [p.clone() for p in params]
            moe.adamw_step(params, [dwg.view(params[0].shape), dwd], step=step, lr=1e-2, master=master, seed=9, **states)
            for p, w, b in zip(params, master, before):
                assert torch.equal(p, w.to(bf16)) and p.isfinite().all()
                # an expert without rows has no gradient: the decay alone moves its weights
                assert torch.equal(p[1], (w[1]).to(bf16)) and (p[[0, 2, 3]] != b[[0, 2, 3]]).float().mean() > 0.5
        assert not states["m"][0][1].view(torch.uint8).any()


def test_with_the_layers_routing(torch, moe):
    """Offsets as the layer's regroup leaves them feed the products."""
    import synth
    from gpu_util import GpuLayer
    case = synth.make_case("tiny_q8")
    s = case.shape
    gpu = GpuLayer(s, case.weights)
    res = gpu.run(case.hidden)
    offsets = torch.from_numpy(res["offsets"]).cuda()
    perm = torch.from_numpy(res["perm"]).long().cuda()
    rows = gpu.hidden(case.hidden)[perm // s.top_k]
    w = torch.randn(s.num_experts, 2, 144, s.d_model, device="cuda").to(torch.bfloat16)
    wq, ws = moe.quantize_blocks(w, tiles=True)
    codes, scale = moe.quantize_blocks(rows)
    h = moe.fp8_gated(codes, scale, wq, ws, offsets)
    for e in range(s.num_experts):
        b, t = int(res["offsets"][e]), int(res["offsets"][e + 1])
        if t > b:
            alone = moe.fp8_gated(codes[b:t], scale[:, b:t], wq[e], ws[e])
            # the same waves' parts of the same sums, but for the split of longer contractions: none here
            assert torch.equal(h[b:t], alone)
