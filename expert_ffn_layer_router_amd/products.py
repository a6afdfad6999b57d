"""Grouped products of expert feed-forward blocks (include/moe_ops.h): 8-bit
codes for serving, 16-bit weights forward and backward for training.

Rows of one expert stand together: group e owns rows offsets[e] ..
offsets[e + 1] - 1 (int32, on the device; `MoeLayer.routing(...)["offsets"]` is
such an array), and `w[e]` is its weight matrix, [n, k] as in torch.nn.Linear.
Without `offsets` there is one group of all rows and w may be [n, k].  Rows
outside every group are not read, and their outputs are left as they were (in
a result that the call allocates: unspecified).

Row matrices may have any row stride that is a multiple of 8 elements (16 for
a product's codes); weights, scales and offsets are contiguous.  A call runs on `stream`
(default: the current stream of the tensors' device) and allocates what it is
not given there; with `out` and `workspace` given it allocates nothing.  On
another stream than the current one the caller orders the call after what
wrote its inputs; their memory is kept from reuse until it is done.  Nothing is
recorded for autograd: the backward calls are the caller's, and with gradients
enabled a tensor that requires one is refused (its result would be cut off).
A given result counts as modified in place: autograd refuses a backward pass
through what it held before."""

from __future__ import annotations

import ctypes
from functools import lru_cache

from . import _lib

ACTIVATIONS = {"silu": _lib.MOE_ACT_SILU, "gelu": _lib.MOE_ACT_GELU}


class _Torch:
    """What the calls need of torch, looked up once (a small product is bound by
    the host, where each of these lookups would show)."""

    def __init__(self):
        import torch
        self.torch = torch
        self.int8, self.float32, self.int32, self.bfloat16 = torch.int8, torch.float32, torch.int32, torch.bfloat16
        self.e4m3, self.e5m2 = torch.float8_e4m3fn, torch.float8_e5m2
        self.types = {torch.bfloat16: _lib.MOE_TYPE_BF16, torch.float16: _lib.MOE_TYPE_FP16,
                      torch.float32: _lib.MOE_TYPE_FP32}
        self.current_device = torch.cuda.current_device
        self.grad_enabled = torch.is_grad_enabled
        # the raw handle without a Stream object around it (2 us less), where this torch has it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
        # autograd then refuses a backward pass through what stood in a tensor (or a list of them) before the call
        self.overwritten = torch.autograd.graph.increment_version
        self.lib = _lib.load()


@lru_cache(maxsize=None)
def _env():
    return _Torch()


def _fits(**sizes):
    """Refuses sizes that the C interface's int32 would cut to their low bits."""
    for name, size in sizes.items():
        if not -(1 << 31) <= size < 1 << 31:
            raise _lib.MoeError(_lib.MOE_ERR_UNSUPPORTED_SHAPE, f"{name}={size} is out of range")


@lru_cache(maxsize=1024)
def _shape(op: int, rows: int, n: int, k: int, groups: int, type_: int, act: int):
    """(the C struct, workspace bytes) of a call: pure host arithmetic of its arguments."""
    _fits(rows=rows, n=n, k=k, groups=groups)
    p = _lib.MoeProduct(rows, n, k, groups, type_, act)
    need = ctypes.c_size_t()
    _lib.check(_lib.load().moe_product_workspace(ctypes.byref(p), op, ctypes.byref(need)))
    return p, need.value


def product_workspace(op: str, rows: int, n: int, k: int, groups: int = 1, dtype=None, activation=None) -> int:
    """Bytes of workspace of a call of `op` ("int8_product", "int8_gated", "expert_product",
    "expert_product_backward", "gated_product" or "gated_product_backward") with this shape."""
    if op not in _lib.MOE_OPS:
        raise ValueError(f"op must be one of {sorted(_lib.MOE_OPS)}, not {op!r}")
    return _shape(_lib.MOE_OPS[op], int(rows), int(n), int(k), int(groups),
                  _type(dtype or _env().bfloat16), _act(activation) if "gated" in op else 0)[1]


def _type(dtype) -> int:
    t = _env().types.get(dtype)
    if t is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return t


def _act(name) -> int:
    a = ACTIVATIONS.get(name or "silu")
    if a is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, not {name!r}")
    return a


class _Call:
    """Checks the tensors of one call against each other, finds its stream and
    makes the calling thread's device and stream match while it allocates and
    enqueues.  (Short calls are bound by the host: the checks are ordered so
    that what is right costs one comparison each.)"""

    __slots__ = ("env", "lib", "index", "guards", "stream", "like", "other")

    def __init__(self, first, stream):
        env = self.env = _env()
        self.lib = env.lib
        self.like = first
        index = self.index = first.get_device()
        if index < 0:
            raise ValueError("the tensors must be on a GPU")
        self.guards = ()
        if env.current_device() != index:
            self.guards = (env.torch.cuda.device(index),)
        self.other = None
        if stream is None:
            self.stream = env.raw_stream(index)
        else:
            if stream.device != first.device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
            self.guards += (env.torch.cuda.stream(stream),)
            self.stream = stream.cuda_stream
            if self.stream != env.raw_stream(index):
                self.other = stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)

    def empty(self, shape, dtype):
        return self.like.new_empty(shape, dtype=dtype)

    def rows(self, name, t, rows, width, dtype):
        """(pointer, row stride) of a [rows, width] matrix."""
        if t.shape != (rows, width) or t.dtype is not dtype or t.get_device() != self.index:
            self.refuse(name, t, (rows, width), dtype)
        if t.requires_grad and self.env.grad_enabled():
            self.refuse_tracked(name)
        stride, one = t.stride()
        if one != 1 and width != 1:
            raise ValueError(f"the values of a row of {name} must be contiguous")
        if self.other is not None:
            t.record_stream(self.other)
        return t.data_ptr(), (stride if rows > 1 else width)

    def plain(self, name, t, shape, dtype):
        """Pointer of a contiguous tensor."""
        if t.shape != shape or t.dtype is not dtype or t.get_device() != self.index:
            self.refuse(name, t, shape, dtype)
        if t.requires_grad and self.env.grad_enabled():
            self.refuse_tracked(name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if self.other is not None:
            t.record_stream(self.other)
        return t.data_ptr()

    def refuse(self, name, t, shape, dtype):
        if t.get_device() != self.index:
            raise ValueError(f"{name} is on {t.device}, not on {self.like.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")

    def refuse_tracked(self, name):
        raise ValueError(f"{name} requires a gradient, and this call records nothing for autograd: call it under "
                         "torch.no_grad() or from a torch.autograd.Function, and its backward call there")

    def offsets(self, offsets, groups):
        if offsets is None:
            return None
        return self.plain("offsets", offsets, (groups + 1,), self.env.int32)

    def workspace(self, workspace, need):
        """(pointer, bytes, tensor kept alive until the call returns)."""
        if workspace is None:
            if need == 0:
                return None, 0, None
            workspace = self.empty(need, self.env.torch.uint8)
        else:
            if workspace.get_device() != self.index:
                raise ValueError(f"workspace is on {workspace.device}, not on {self.like.device}")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
            if self.other is not None:
                workspace.record_stream(self.other)
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace

    def result(self, name, out, rows, width, dtype):
        if out is None:
            out = self.empty((rows, width), dtype)
            return out, out.data_ptr(), width
        pointer, stride = self.rows(name, out, rows, width, dtype)
        self.env.overwritten(out)
        return out, pointer, stride

    def plain_result(self, name, out, shape, dtype):
        """(a contiguous result, its pointer)."""
        if out is None:
            out = self.empty(shape, dtype)
            return out, out.data_ptr()
        pointer = self.plain(name, out, shape, dtype)
        self.env.overwritten(out)
        return out, pointer


def _weights(w, gated):
    """(groups, n, k) of w [groups, n (gated: 2n), k] or [n, k]."""
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [groups, n, k] or [n, k], not {list(w.shape)}")
    groups = w.shape[0] if w.dim() == 3 else 1
    wide, k = w.shape[-2], w.shape[-1]
    if gated and wide % 2:
        raise ValueError(f"w has {wide} rows a group; gate and up rows come in equal numbers")
    return groups, wide // 2 if gated else wide, k


def _matrix_rows(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, not {list(t.shape)}")
    return t.shape[0]


def quantize_rows(x, codes=None, scale=None, stream=None):
    """(codes int8 [rows, k], scale fp32 [rows]) of x [rows, k] (bf16 or fp16):
    scale = max|row| / 127, codes = rint(row / scale) (moe_quantize_rows)."""
    rows = _matrix_rows("x", x)
    k = x.shape[1]
    if rows | k > 0x7FFFFFFF:
        _fits(rows=rows, k=k)
    with _Call(x, stream) as c:
        px, ldx = c.rows("x", x, rows, k, x.dtype)
        codes, pc, ldc = c.result("codes", codes, rows, k, c.env.int8)
        scale, ps = c.plain_result("scale", scale, (rows,), c.env.float32)
        _lib.check(c.lib.moe_quantize_rows(rows, k, _type(x.dtype), px, ldx, pc, ldc, ps, c.stream))
    return codes, scale


def _int8(op, codes, scale, w, w_scale, offsets, activation, out, dtype, workspace, stream):
    gated = activation is not None
    rows = _matrix_rows("codes", codes)
    groups, n, k = _weights(w, gated)
    if dtype is None:
        dtype = out.dtype if out is not None else _env().bfloat16
    with _Call(codes, stream) as c:
        pc, ldc = c.rows("codes", codes, rows, k, c.env.int8)
        ps = c.plain("scale", scale, (rows,), c.env.float32)
        pw = c.plain("w", w, w.shape, c.env.int8)
        pws = c.plain("w_scale", w_scale, w.shape[:-1], c.env.float32)
        po = c.offsets(offsets, groups)
        shape, need = _shape(op, rows, n, k, groups, _type(dtype), _act(activation) if gated else 0)
        out, pout, ldout = c.result("out", out, rows, n, dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        fn = c.lib.moe_int8_gated if gated else c.lib.moe_int8_product
        _lib.check(fn(ctypes.byref(shape), pc, ldc, ps, pw, pws, po, pout, ldout, ws, ws_bytes, c.stream))
    return out


def int8_product(codes, scale, w, w_scale, offsets=None, out=None, dtype=None, workspace=None, stream=None):
    """y[r] = scale[r] w_scale[e] * (codes[r] w[e]^T): codes int8 [rows, k], scale fp32 [rows],
    w int8 [groups, n, k], w_scale fp32 [groups, n]; y [rows, n] bf16 (default), fp16 or fp32."""
    return _int8(_lib.MOE_OPS["int8_product"], codes, scale, w, w_scale, offsets, None, out, dtype, workspace, stream)


def int8_gated(codes, scale, w, w_scale, offsets=None, activation="silu", out=None, dtype=None, workspace=None,
               stream=None):
    """h = act(g) * u, (g, u) the int8 product with w int8 [groups, 2n, k] (gate rows, then up rows);
    h [rows, n] bf16 (default) or fp16."""
    return _int8(_lib.MOE_OPS["int8_gated"], codes, scale, w, w_scale, offsets, activation or "silu", out, dtype,
                 workspace, stream)


def expert_product(x, w, offsets=None, out=None, workspace=None, stream=None):
    """y = x w[e]^T: x [rows, k], w [groups, n, k], both bf16 or both fp16; y [rows, n]."""
    rows = _matrix_rows("x", x)
    groups, n, k = _weights(w, False)
    with _Call(x, stream) as c:
        px, ldx = c.rows("x", x, rows, k, x.dtype)
        pw = c.plain("w", w, w.shape, x.dtype)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_OPS["expert_product"], rows, n, k, groups, _type(x.dtype), 0)
        out, pout, ldout = c.result("out", out, rows, n, x.dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_expert_product(ctypes.byref(shape), px, ldx, pw, po, pout, ldout, ws, ws_bytes, c.stream))
    return out


def gated_product(x, w, offsets=None, activation="silu", save=False, out=None, gate_up=None, workspace=None,
                  stream=None):
    """h = act(g) * u with (g, u) = x w[e]^T: w [groups, 2n, k] (gate rows, then up rows); h [rows, n].
    With `save` (or a `gate_up` to fill) returns (h, gate_up [rows, 2n]), which the backward pass takes."""
    rows = _matrix_rows("x", x)
    groups, n, k = _weights(w, True)
    save = save or gate_up is not None
    with _Call(x, stream) as c:
        px, ldx = c.rows("x", x, rows, k, x.dtype)
        pw = c.plain("w", w, w.shape, x.dtype)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_OPS["gated_product"], rows, n, k, groups, _type(x.dtype), _act(activation))
        out, pout, ldout = c.result("out", out, rows, n, x.dtype)
        pg, ldg = None, 0
        if save:
            gate_up, pg, ldg = c.result("gate_up", gate_up, rows, 2 * n, x.dtype)
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        _lib.check(c.lib.moe_gated_product(ctypes.byref(shape), px, ldx, pw, po, pout, ldout, pg, ldg, ws, ws_bytes,
                                           c.stream))
    return (out, gate_up) if save else out


def _backward(name, dy, gate_up, x, w, offsets, activation, need_dx, need_dw, dx, dw, dw_dtype, workspace, stream):
    gated = activation is not None
    rows = _matrix_rows("dh" if gated else "dy", dy)
    dtype = dy.dtype
    need_dx, need_dw = need_dx or dx is not None, need_dw or dw is not None
    if x is None and need_dw:
        raise ValueError("x is needed for dw")
    if w is not None:
        groups, n, k = _weights(w, gated)
        w_shape = w.shape
    else:
        if need_dx or x is None:
            raise ValueError("w is needed for dx" if need_dx else "x or w is needed")
        _matrix_rows("x", x)
        n, k = dy.shape[1], x.shape[1]
        groups = 1 if offsets is None else offsets.numel() - 1
        w_shape = (groups, 2 * n if gated else n, k)
        if offsets is None and (dw is None or dw.dim() == 2):
            w_shape = w_shape[1:]
    with _Call(dy, stream) as c:
        py, ldy = c.rows("dh" if gated else "dy", dy, rows, n, dtype)
        px, ldx = (None, 0) if x is None else c.rows("x", x, rows, k, dtype)
        pw = None if w is None else c.plain("w", w, w_shape, dtype)
        po = c.offsets(offsets, groups)
        shape, need = _shape(_lib.MOE_OPS[name], rows, n, k, groups, _type(dtype), _act(activation) if gated else 0)
        pdx, lddx, pdw = None, 0, None
        if need_dx:
            dx, pdx, lddx = c.result("dx", dx, rows, k, dtype)
        if need_dw:
            dw, pdw = c.plain_result("dw", dw, w_shape, dw_dtype or (dtype if dw is None else dw.dtype))
        ws, ws_bytes, _alive = c.workspace(workspace, need)
        dw_type = _type(dw.dtype) if need_dw else shape.type
        head = (ctypes.byref(shape), py, ldy)
        tail = (px, ldx, pw, po, pdx, lddx, pdw, dw_type, ws, ws_bytes, c.stream)
        if gated:
            pg, ldg = c.rows("gate_up", gate_up, rows, 2 * n, dtype)
            _lib.check(c.lib.moe_gated_product_backward(*head, pg, ldg, *tail))
        else:
            _lib.check(c.lib.moe_expert_product_backward(*head, *tail))
    return dx, dw


def expert_product_backward(dy, x, w, offsets=None, need_dx=True, need_dw=True, dx=None, dw=None, dw_dtype=None,
                            workspace=None, stream=None):
    """(dx, dw) of expert_product for the gradient dy [rows, n]: dx = dy w[e], dw[e] = dy_e^T x_e (of w's
    dtype, or `dw_dtype` fp32; zero for a group without rows).  What is not needed is None.  x may be None
    without dw, w without dx (dw is then [groups, n, k], or [n, k] without offsets)."""
    return _backward("expert_product_backward", dy, None, x, w, offsets, None, need_dx, need_dw, dx, dw, dw_dtype,
                     workspace, stream)


def gated_product_backward(dh, gate_up, x, w, offsets=None, activation="silu", need_dx=True, need_dw=True, dx=None,
                           dw=None, dw_dtype=None, workspace=None, stream=None):
    """(dx, dw) of gated_product for the gradient dh [rows, n] and the gate_up it saved; the rest as for
    expert_product_backward."""
    return _backward("gated_product_backward", dh, gate_up, x, w, offsets, activation or "silu", need_dx, need_dw, dx,
                     dw, dw_dtype, workspace, stream)
