"""Grouped products of expert feed-forward blocks in 8-bit floating point
(include/moe_fp8.h): e4m3 codes with a fp32 scale for each block of 128, for
serving and, with the backward calls, for training.

Codes are torch.float8_e4m3fn.  Rows have a scale for each 128 of their values,
block by block: scale [ceil(k / 128), rows].  Weights have one for each
128 x 128: w [groups, n, k] and w_scale [groups, ceil(n / 128), ceil(k / 128)];
the gated block's are w [groups, 2, n, k] (gate, up) and w_scale [groups, 2,
...].  Without `offsets` there is one group of all rows and the groups'
dimension may be left out.  n and k are multiples of 16.

What products.py says of groups, strides, streams, workspaces and gradients
holds here.  The rows of scale may have any stride of at least `rows`.  The
weights' gradient is taken in 16 bits: expert_product_backward(dy, x, None,
offsets, need_dx=False), for the gated block with the slopes that
fp8_gated_backward returns as dy."""

from __future__ import annotations

import ctypes
from functools import lru_cache

from . import _lib
from .products import _act, _Call, _env, _fits, _matrix_rows, _type

BLOCK = 128  # values that share a scale


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


@lru_cache(maxsize=1024)
def _shape(op: int, rows: int, n: int, k: int, groups: int, type_: int, act: int):
    """(the C struct, workspace bytes) of a call: pure host arithmetic of its arguments."""
    _fits(rows=rows, n=n, k=k, groups=groups)
    p = _lib.MoeProduct(rows, n, k, groups, type_, act)
    need = ctypes.c_size_t()
    _lib.check(_lib.load().moe_fp8_workspace(ctypes.byref(p), op, ctypes.byref(need)))
    return p, need.value


def fp8_workspace(op: str, rows: int, n: int, k: int, groups: int = 1, dtype=None, activation=None) -> int:
    """Bytes of workspace of a call of `op` ("fp8_product", "fp8_gated", "fp8_product_backward" or
    "fp8_gated_backward") with this shape."""
    if op not in _lib.MOE_FP8_OPS:
        raise ValueError(f"op must be one of {sorted(_lib.MOE_FP8_OPS)}, not {op!r}")
    return _shape(_lib.MOE_FP8_OPS[op], int(rows), int(n), int(k), int(groups),
                  _type(dtype or _env().bfloat16), _act(activation) if "gated" in op else 0)[1]


def _weights(w, gated):
    """(groups, n, k) of w [groups, n, k] or [n, k] (gated: [groups, 2, n, k] or [2, n, k])."""
    if gated:
        if w.dim() not in (3, 4) or w.shape[-3] != 2:
            raise ValueError(f"w must be [groups, 2, n, k] or [2, n, k], not {list(w.shape)}")
        return (w.shape[0] if w.dim() == 4 else 1), w.shape[-2], w.shape[-1]
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [groups, n, k] or [n, k], not {list(w.shape)}")
    return (w.shape[0] if w.dim() == 3 else 1), w.shape[-2], w.shape[-1]


def _operands(c, codes, scale, w, w_scale, rows, width):
    """(codes, their stride, scale, its stride, w, w_scale) as pointers."""
    env = c.env
    e4m3 = env.e4m3
    shape = w.shape
    pc, ldc = c.rows("codes", codes, rows, width, e4m3)
    ps, lds = c.rows("scale", scale, (width + 127) // BLOCK, rows, env.float32)
    pw = c.plain("w", w, shape, e4m3)
    pws = c.plain("w_scale", w_scale, _scale_shape(shape), env.float32)
    return pc, ldc, ps, lds, pw, pws


@lru_cache(maxsize=1024)
def _scale_shape(shape):
    return (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]))


def quantize_blocks(x, tiles=False, codes=None, scale=None, stream=None):
    """(codes, scale) of x (bf16 or fp16): scale = max|block| / 448, codes = x / scale rounded to e4m3.
    Rows x [rows, k] have blocks of 128 of a row's values, scale [ceil(k / 128), rows]
    (moe_quantize_blocks).  With `tiles`, weights x [..., n, k] have blocks of 128 x 128, scale
    [..., ceil(n / 128), ceil(k / 128)] (moe_quantize_tiles; x, codes and scale contiguous): the gated
    block's as [groups, 2, n, k]."""
    e4m3 = _env().e4m3
    if not tiles:
        rows = _matrix_rows("x", x)
        k = x.shape[1]
        if rows | k > 0x7FFFFFFF:
            _fits(rows=rows, k=k)
        with _Call(x, stream) as c:
            px, ldx = c.rows("x", x, rows, k, x.dtype)
            codes, pc, ldc = c.result("codes", codes, rows, k, e4m3)
            scale, ps, lds = c.result("scale", scale, _blocks(k), rows, c.env.float32)
            _lib.check(c.lib.moe_quantize_blocks(rows, k, _type(x.dtype), px, ldx, pc, ldc, ps, lds,
                                                 c.stream))
        return codes, scale
    if x.dim() < 2:
        raise ValueError(f"x must be [..., n, k], not {list(x.shape)}")
    n, k = x.shape[-2:]
    matrices = x[..., 0, 0].numel() if n and k else 0
    _fits(matrices=matrices, n=n, k=k)
    shape = _scale_shape(x.shape)
    with _Call(x, stream) as c:
        px = c.plain("x", x, x.shape, x.dtype)
        codes, pc = c.plain_result("codes", codes, x.shape, e4m3)
        scale, ps = c.plain_result("scale", scale, shape, c.env.float32)
        _lib.check(c.lib.moe_quantize_tiles(matrices, n, k, _type(x.dtype), px, pc, ps, c.stream))
    return codes, scale


def fp8_product(codes, scale, w, w_scale, offsets=None, out=None, dtype=None, workspace=None, stream=None):
    """y = x w[e]^T of rows and weights in codes: codes [rows, k], scale [ceil(k / 128), rows],
    w [groups, n, k], w_scale [groups, ceil(n / 128), ceil(k / 128)]; y [rows, n] bf16 (default) or fp16."""
    rows = _matrix_rows("codes", codes)
    groups, n, k = _weights(w, False)
    if dtype is None:
        dtype = out.dtype if out is not None else _env().bfloat16
    with _Call(codes, stream) as c:
        operands = _operands(c, codes, scale, w, w_scale, rows, k)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_FP8_OPS["fp8_product"], rows, n, k, groups, _type(dtype), 0)
        out, pout, ldout = c.result("out", out, rows, n, dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_fp8_product(ctypes.byref(shape), *operands, po, pout, ldout, ws, ws_bytes, c.stream))
    return out


def fp8_gated(codes, scale, w, w_scale, offsets=None, activation="silu", save=False, out=None, gate_up=None, dtype=None,
              workspace=None, stream=None):
    """h = act(g) * u, g and u the products with w[e, 0] and w[e, 1]: w [groups, 2, n, k], w_scale
    [groups, 2, ceil(n / 128), ceil(k / 128)]; h [rows, n] bf16 (default) or fp16.  With `save` (or a `gate_up`
    to fill) returns (h, gate_up [rows, 2n]), which the backward pass takes."""
    rows = _matrix_rows("codes", codes)
    groups, n, k = _weights(w, True)
    save = save or gate_up is not None
    if dtype is None:
        dtype = out.dtype if out is not None else gate_up.dtype if gate_up is not None else _env().bfloat16
    with _Call(codes, stream) as c:
        operands = _operands(c, codes, scale, w, w_scale, rows, k)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_FP8_OPS["fp8_gated"], rows, n, k, groups, _type(dtype), _act(activation))
        out, pout, ldout = c.result("out", out, rows, n, dtype)
        pg, ldg = None, 0
        if save:
            gate_up, pg, ldg = c.result("gate_up", gate_up, rows, 2 * n, dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_fp8_gated(ctypes.byref(shape), *operands, po, pout, ldout, pg, ldg, ws, ws_bytes,
                                       c.stream))
    return (out, gate_up) if save else out


def fp8_product_backward(codes, scale, w, w_scale, offsets=None, dx=None, dtype=None, workspace=None, stream=None):
    """dx = dy w[e] of fp8_product for the gradient dy in codes [rows, n] with scale [ceil(n / 128), rows]
    (quantize_blocks of dy); dx [rows, k] bf16 (default) or fp16."""
    rows = _matrix_rows("codes", codes)
    groups, n, k = _weights(w, False)
    if dtype is None:
        dtype = dx.dtype if dx is not None else _env().bfloat16
    with _Call(codes, stream) as c:
        operands = _operands(c, codes, scale, w, w_scale, rows, n)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_FP8_OPS["fp8_product_backward"], rows, n, k, groups, _type(dtype), 0)
        dx, pdx, lddx = c.result("dx", dx, rows, k, dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_fp8_product_backward(ctypes.byref(shape), *operands, po, pdx, lddx, ws, ws_bytes,
                                                  c.stream))
    return dx


def fp8_gated_backward(dh, gate_up, w, w_scale, offsets=None, activation="silu", need_dx=True, need_slopes=True,
                       dx=None, slopes=None, workspace=None, stream=None):
    """(dx, slopes) of fp8_gated for the gradient dh [rows, n] and the gate_up it saved (both bf16 or fp16, as are
    dx [rows, k] and slopes [rows, 2n]): slopes = (dg, du), which go through codes into dx = dg w[e, 0] + du w[e, 1].
    What is not needed is None."""
    rows = _matrix_rows("dh", dh)
    groups, n, k = _weights(w, True)
    dtype = dh.dtype
    need_dx, need_slopes = need_dx or dx is not None, need_slopes or slopes is not None
    with _Call(dh, stream) as c:
        pd, ldd = c.rows("dh", dh, rows, n, dtype)
        pg, ldg = c.rows("gate_up", gate_up, rows, 2 * n, dtype)
        pw = c.plain("w", w, w.shape, c.env.e4m3)
        pws = c.plain("w_scale", w_scale, _scale_shape(w.shape), c.env.float32)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_FP8_OPS["fp8_gated_backward"], rows, n, k, groups, _type(dtype),
                             _act(activation))
        pdx, lddx, psl, ldsl = None, 0, None, 0
        if need_dx:
            dx, pdx, lddx = c.result("dx", dx, rows, k, dtype)
        if need_slopes:
            slopes, psl, ldsl = c.result("slopes", slopes, rows, 2 * n, dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_fp8_gated_backward(ctypes.byref(shape), pd, ldd, pg, ldg, pw, pws, po, pdx, lddx, psl,
                                                ldsl, ws, ws_bytes, c.stream))
    return dx, slopes
