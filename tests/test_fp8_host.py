"""Host-only tests of the products in 8-bit floating point and of AdamW: what
the C ABI and the binding refuse before anything is enqueued.  Nothing here
launches a kernel."""

import ctypes
import os

import pytest

from expert_ffn_layer_router_amd import _lib

FAKE = 0x10000  # an aligned address that validation never dereferences
BF16, FP16, FP32 = _lib.MOE_TYPE_BF16, _lib.MOE_TYPE_FP16, _lib.MOE_TYPE_FP32
INVALID, SHAPE, SMALL = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED_SHAPE, _lib.MOE_ERR_WORKSPACE_TOO_SMALL
OPS = _lib.MOE_FP8_OPS


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from expert_ffn_layer_router_amd import build
        build.build()
    return _lib.load()


def shape(**kw):
    base = dict(rows=0, n=64, k=64, groups=1, type=BF16, activation=0)
    base.update(kw)
    return _lib.MoeProduct(**base)


def workspace(lib, op, **kw):
    n = ctypes.c_size_t()
    st = lib.moe_fp8_workspace(ctypes.byref(shape(**kw)), OPS[op], ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("op", sorted(OPS))
@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=(1 << 22) + 1), dict(n=0), dict(n=24), dict(n=65552),
                                dict(k=0), dict(k=8), dict(k=24), dict(k=65552), dict(groups=0), dict(groups=257),
                                dict(type=FP32), dict(type=3), dict(type=-1), dict(activation=2), dict(activation=-1)])
def test_shapes_refused(lib, op, kw):
    assert workspace(lib, op, **kw)[0] == SHAPE, _lib.last_error()


def test_shapes_by_operator(lib):
    for op in ("fp8_gated", "fp8_gated_backward"):
        assert workspace(lib, op, n=32768)[0] == 0
        assert workspace(lib, op, n=32784)[0] == SHAPE
        assert workspace(lib, op, activation=1)[0] == 0
    for op in ("fp8_product", "fp8_product_backward"):
        assert workspace(lib, op, n=65536)[0] == 0
        assert workspace(lib, op, activation=1)[0] == SHAPE
    n = ctypes.c_size_t()
    assert lib.moe_fp8_workspace(None, 0, ctypes.byref(n)) == INVALID
    assert lib.moe_fp8_workspace(ctypes.byref(shape()), 4, ctypes.byref(n)) == INVALID
    assert lib.moe_fp8_workspace(ctypes.byref(shape()), -1, ctypes.byref(n)) == INVALID
    assert lib.moe_fp8_workspace(ctypes.byref(shape()), 0, None) == INVALID


def test_workspace_holds_the_slopes_and_the_parts(lib):
    # codes of (dg, du) in whole blocks, and a scale for each
    st, n = workspace(lib, "fp8_gated_backward", rows=1000, n=4000, k=4096)
    assert st == 0 and n >= 1000 * 2 * 4096 + 1000 * 2 * 32 * 4
    # long sums and few tiles: the contraction is split
    assert workspace(lib, "fp8_product", rows=2000, n=1024, k=8192)[1] > 0
    assert workspace(lib, "fp8_product_backward", rows=1000, n=8192, k=256)[1] > 0
    # sums too short to split, few rows, none
    assert workspace(lib, "fp8_product", rows=4096, n=8192, k=256) == (0, 0)
    assert workspace(lib, "fp8_product", rows=8, n=128, k=8192) == (0, 0)
    for op in OPS:
        assert workspace(lib, op, rows=0, n=128, k=8192) == (0, 0)
        for kw in (dict(rows=1000, n=256, k=8192), dict(rows=77, groups=256), dict(rows=5000, n=4096, k=4096)):
            assert workspace(lib, op, type=BF16, **kw) == workspace(lib, op, type=FP16, **kw)
    # the largest shapes stay in range of the size type
    st, n = workspace(lib, "fp8_gated_backward", rows=1 << 22, n=32768, k=65536, groups=256)
    assert st == 0 and n >= (1 << 22) * 65536


def product(lib, op, **over):
    """A call that fails validation or has no rows (never launches)."""
    fields = {f: over.pop(f) for f in list(over) if f in dict(_lib.MoeProduct._fields_)}
    p = shape(**fields)
    back = op.endswith("backward")
    a = dict(codes=FAKE, ldc=p.n if back else p.k, scale=FAKE, lds=max(p.rows, 0), w=FAKE, w_scale=FAKE, offsets=None,
             out=FAKE, ldout=p.k if back else p.n, gate_up=None, ldgu=2 * p.n, ws=FAKE, ws_bytes=1 << 40)
    a.update(over)
    head = (ctypes.byref(p), a["codes"], a["ldc"], a["scale"], a["lds"], a["w"], a["w_scale"], a["offsets"], a["out"],
            a["ldout"])
    keep = (a["gate_up"], a["ldgu"]) if op == "fp8_gated" else ()
    return getattr(lib, "moe_" + op)(*head, *keep, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("op", ["fp8_product", "fp8_gated", "fp8_product_backward"])
def test_product_arguments_refused(lib, op):
    assert product(lib, op) == 0  # no rows: nothing to do
    assert product(lib, op, codes=None, scale=None, out=None) == 0
    for kw in (dict(codes=None), dict(codes=FAKE + 8), dict(ldc=48), dict(ldc=72), dict(ldc=(1 << 20) + 16),
               dict(scale=None), dict(scale=FAKE + 2), dict(lds=3), dict(lds=(1 << 22) + 1), dict(w=None),
               dict(w=FAKE + 8), dict(w_scale=None), dict(w_scale=FAKE + 2), dict(out=None), dict(out=FAKE + 4),
               dict(ldout=56), dict(ldout=68), dict(groups=2), dict(groups=2, offsets=FAKE + 2)):
        assert product(lib, op, rows=4, **kw) == INVALID, kw
    sizes = dict(rows=1000, n=8192, k=256) if op == "fp8_product_backward" else dict(rows=2000, n=1024, k=8192)
    assert product(lib, op, ws_bytes=1, **sizes) == SMALL
    assert "needs" in _lib.last_error()
    assert product(lib, op, ws=None, **sizes) == INVALID
    assert product(lib, op, ws=FAKE + 8, **sizes) == INVALID
    if op == "fp8_gated":
        assert product(lib, op, rows=4, gate_up=FAKE, ldgu=64) == INVALID
        assert product(lib, op, rows=4, gate_up=FAKE + 8) == INVALID


def test_gated_backward_arguments_refused(lib):
    def call(**over):
        fields = {f: over.pop(f) for f in list(over) if f in dict(_lib.MoeProduct._fields_)}
        p = shape(**fields)
        a = dict(dh=FAKE, lddh=p.n, gu=FAKE, ldgu=2 * p.n, w=FAKE, w_scale=FAKE, offsets=None, dx=FAKE, lddx=p.k,
                 slopes=FAKE, ldsl=2 * p.n, ws=FAKE, ws_bytes=1 << 40)
        a.update(over)
        return lib.moe_fp8_gated_backward(ctypes.byref(p), a["dh"], a["lddh"], a["gu"], a["ldgu"], a["w"], a["w_scale"],
                                          a["offsets"], a["dx"], a["lddx"], a["slopes"], a["ldsl"], a["ws"],
                                          a["ws_bytes"], None)

    assert call() == 0
    assert call(dh=None, gu=None, dx=None, slopes=None, ws=None, ws_bytes=0) == 0
    assert call(rows=4, dx=None, slopes=None, w=None, w_scale=None) == 0  # nothing asked for
    for kw in (dict(dh=None), dict(dh=FAKE + 8), dict(lddh=56), dict(lddh=68), dict(gu=None), dict(ldgu=64), dict(w=None),
               dict(w_scale=None), dict(dx=FAKE + 8), dict(lddx=56), dict(slopes=FAKE + 8), dict(ldsl=64),
               dict(groups=3), dict(ws=None), dict(ws=FAKE + 8)):
        assert call(rows=4, **kw) == INVALID, kw
    assert call(rows=4, ws_bytes=8) == SMALL


def test_quantize_arguments_refused(lib):
    def rows(rows=4, k=64, type_=BF16, x=FAKE, ldx=64, codes=FAKE, ldc=64, scale=FAKE, lds=4):
        return lib.moe_quantize_blocks(rows, k, type_, x, ldx, codes, ldc, scale, lds, None)

    assert rows(rows=0) == 0
    assert rows(rows=0, x=None, codes=None, scale=None, lds=0) == 0
    for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(k=0), dict(k=8), dict(k=24), dict(k=65552), dict(type_=FP32)):
        assert rows(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(x=FAKE + 2), dict(ldx=56), dict(ldx=68), dict(codes=None), dict(codes=FAKE + 8),
               dict(ldc=48), dict(ldc=72), dict(scale=None), dict(scale=FAKE + 2), dict(lds=3)):
        assert rows(**kw) == INVALID, kw

    def tiles(matrices=2, n=64, k=64, type_=BF16, x=FAKE, codes=FAKE, scale=FAKE):
        return lib.moe_quantize_tiles(matrices, n, k, type_, x, codes, scale, None)

    assert tiles(matrices=0, x=None, codes=None, scale=None) == 0
    for kw in (dict(matrices=-1), dict(matrices=513), dict(n=0), dict(n=-16), dict(n=65537), dict(k=0), dict(k=24),
               dict(type_=FP32)):
        assert tiles(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(x=FAKE + 8), dict(codes=None), dict(codes=FAKE + 8), dict(scale=None),
               dict(scale=FAKE + 2)):
        assert tiles(**kw) == INVALID, kw


def adamw(lib, tensors=(), **over):
    n = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0, seed=0, step=1, state_bits=32)
    n.update(over)
    table = (_lib.MoeAdamwTensor * max(1, len(tensors)))(*tensors)
    return lib.moe_adamw_step(ctypes.byref(_lib.MoeAdamw(**n)), len(tensors), table, None)


def tensor(at=FAKE, count=0, **over):
    """A tensor whose arrays lie 1 MiB apart."""
    far = 1 << 20
    t = dict(param=at, grad=at + far, m=at + 2 * far, v=at + 3 * far, count=count, param_type=BF16, grad_type=BF16)
    t.update(over)
    return _lib.MoeAdamwTensor(**t)


def test_adamw_refusals(lib):
    nan, inf = float("nan"), float("inf")
    assert adamw(lib) == 0
    assert adamw(lib, [tensor()]) == 0  # no values: nothing to do
    assert adamw(lib, [tensor(param=None, grad=None, m=None, v=None)]) == 0
    for kw in (dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=nan),
               dict(eps=-1e-8), dict(eps=nan), dict(eps=inf), dict(weight_decay=inf), dict(step=0), dict(step=-1),
               dict(device_lr=FAKE + 2), dict(device_step=FAKE + 1), dict(device_grad_scale=FAKE + 2)):
        assert adamw(lib, **kw) == INVALID, kw
    for kw in (dict(state_bits=16), dict(state_bits=0)):
        assert adamw(lib, **kw) == SHAPE, kw
    # numbers on the device take the host's place
    assert adamw(lib, lr=nan, device_lr=FAKE) == 0 and adamw(lib, step=0, device_step=FAKE) == 0
    assert lib.moe_adamw_step(None, 0, None, None) == INVALID
    n = _lib.MoeAdamw(beta1=0.9, beta2=0.9, step=1, state_bits=32)
    assert lib.moe_adamw_step(ctypes.byref(n), -1, None, None) == INVALID
    assert lib.moe_adamw_step(ctypes.byref(n), 1, None, None) == INVALID
    for kw in (dict(count=-1), dict(count=(1 << 35) + 1), dict(count=4, param_type=3), dict(count=4, grad_type=FP16),
               dict(count=4, param_type=FP32)):
        assert adamw(lib, [tensor(**kw)]) == SHAPE, kw
    for name in ("param", "grad", "m", "v"):
        assert adamw(lib, [tensor(count=4, **{name: None})]) == INVALID, name
        assert adamw(lib, [tensor(count=4, **{name: FAKE + (5 << 20) + 8})]) == INVALID, name
    assert adamw(lib, [tensor(count=4, param_type=FP32, grad_type=FP32, master=FAKE + (5 << 20))]) == INVALID
    assert adamw(lib, [tensor(count=4, m_scale=FAKE + (5 << 20))]) == INVALID  # 32 bits
    assert adamw(lib, [tensor(count=4)], state_bits=8) == INVALID               # no scales
    assert adamw(lib, [tensor(count=4, m_scale=FAKE + (5 << 20), v_scale=FAKE + (6 << 20) + 2)], state_bits=8) == INVALID


def test_adamw_refuses_memory_that_a_step_would_race_on(lib):
    a, b = FAKE, FAKE + (16 << 20)
    far = 1 << 20

    def shared(*tensors, **kw):
        status = adamw(lib, list(tensors), **kw)
        assert "share memory" in _lib.last_error() or status == 0, _lib.last_error()
        return status == INVALID

    assert shared(tensor(a, 100), tensor(a, 100))                                      # twice the same
    assert shared(tensor(a, 100), tensor(b, 100, param=a + 96))                        # an end in another's begin
    assert shared(tensor(a, 100, m=a))                                                 # a state over its weights
    assert shared(tensor(a, 100, grad=a + 96))                                         # gradients over the weights
    assert shared(tensor(a, 100), tensor(b, 100, grad=a + 2 * far))                    # another's state as gradients
    assert shared(tensor(a, 100, master=a + 3 * far + 64))
    assert shared(tensor(a, 1000, m_scale=a + 4 * far, v_scale=a + 4 * far + 16), state_bits=8)
    # a long gradient that begins before another tensor's arrays and reaches past their begin
    long = tensor(a + (256 << 20), 4 << 20, grad=a, m=a + (512 << 20), v=a + (768 << 20))
    assert shared(long, tensor(b, 100, grad=a + far, param=a + 4 * far))


def test_binding_refusals():
    import torch

    import expert_ffn_layer_router_amd as moe
    e4m3 = torch.float8_e4m3fn
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, scale = torch.zeros(4, 64, dtype=e4m3), torch.zeros(1, 4)
    w, w_scale = torch.zeros(2, 64, 64, dtype=e4m3), torch.zeros(2, 1, 1)
    for call in (lambda: moe.quantize_blocks(x), lambda: moe.quantize_blocks(x, tiles=True),
                 lambda: moe.fp8_product(codes, scale, w, w_scale), lambda: moe.fp8_gated(codes, scale, w, w_scale),
                 lambda: moe.fp8_product_backward(codes, scale, w, w_scale),
                 lambda: moe.fp8_gated_backward(x, x, w, w_scale),
                 lambda: moe.adamw_step([x], [x], [x], [x], 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="matrix"):
        moe.quantize_blocks(x[0])
    with pytest.raises(ValueError, match="x must be"):
        moe.quantize_blocks(x[0], tiles=True)
    with pytest.raises(ValueError, match="matrix"):
        moe.fp8_product(codes[0], scale, w, w_scale)
    for bad in (w[0, 0], w[None]):
        with pytest.raises(ValueError, match="w must be"):
            moe.fp8_product(codes, scale, bad, w_scale)
    for bad in (w[0], torch.zeros(3, 64, 64, dtype=e4m3)):
        with pytest.raises(ValueError, match="w must be"):
            moe.fp8_gated(codes, scale, bad, w_scale)
    with pytest.raises(ValueError, match="op must be"):
        moe.fp8_workspace("expert_product", 1, 16, 16)
    with pytest.raises(ValueError, match="activation"):
        moe.fp8_workspace("fp8_gated", 1, 16, 16, activation="tanh")
    for bad in (dict(n=24), dict(rows=1 << 31), dict(k=(1 << 32) + 64)):
        with pytest.raises(moe.MoeError) as e:
            moe.fp8_workspace("fp8_product", **{**dict(rows=1, n=16, k=16), **bad})
        assert e.value.status == SHAPE
    for at in (((1 << 32) + 4, 64), (4, (1 << 32) + 64)):
        with pytest.raises(moe.MoeError) as e:  # refused before the device is looked at
            moe.quantize_blocks(torch.empty(1, dtype=torch.bfloat16).expand(at))
        assert e.value.status == SHAPE
    with pytest.raises(ValueError, match="list"):
        moe.adamw_step(x, [x], [x], [x], 1)
    with pytest.raises(ValueError, match="grads has 2"):
        moe.adamw_step([x], [x, x], [x], [x], 1)
    with pytest.raises(ValueError, match="together"):
        moe.adamw_step([x], [x], [x], [x], 1, m_scale=[scale])
    with pytest.raises(ValueError, match="bits"):
        moe.adamw_states([x], bits=16)
    states = moe.adamw_states([x, x[0]], bits=8)
    assert [t.numel() for t in states["m_scale"]] == [2, 1] and states["v"][1].dtype == torch.float8_e5m2
