"""AdamW over many tensors in one call (include/moe_optim.h), with states in 32
or in 8 bits: the step that takes the gradients of the products' backward calls
to new weights.

    states = adamw_states(params, bits=8)             # once
    adamw_step(params, grads, step=t, lr=1e-4, **states)

A call runs on `stream` (default: the current stream of the tensors' device),
updates params, master and the states in place and allocates nothing.  It is
made under torch.no_grad(), as every update of a leaf in place."""

from __future__ import annotations

import ctypes
import struct
from functools import lru_cache
from itertools import chain
from operator import attrgetter, index

from . import _lib
from .products import _Call, _env, _type

_dtype_of, _shape_of, _tracked = attrgetter("dtype"), attrgetter("shape"), attrgetter("requires_grad")
BLOCK = 128  # values of an 8-bit state that share a scale


def adamw_states(params, bits=32):
    """The states of a first step: a dict of m and v (and, with 8 bits, m_scale and v_scale), lists with a
    tensor for each of params."""
    import torch
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, not {bits!r}")

    def zeros(dtype):
        return [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params]

    if bits == 32:
        return {"m": zeros(torch.float32), "v": zeros(torch.float32)}
    states = {"m": zeros(torch.float8_e4m3fn), "v": zeros(torch.float8_e5m2)}
    for name in ("m_scale", "v_scale"):
        states[name] = [torch.zeros((p.numel() + BLOCK - 1) // BLOCK, dtype=torch.float32, device=p.device)
                        for p in params]
    return states


@lru_cache(maxsize=2)
def _tensor_types(none):
    torch = _env().torch
    return frozenset((torch.Tensor, torch.nn.Parameter) + ((type(None),) if none else ()))


def _lists(**lists):
    length = None
    for name, tensors in lists.items():
        if tensors is None:
            continue
        if not isinstance(tensors, (list, tuple)):
            raise ValueError(f"{name} must be a list of tensors")
        if length is None:
            length = len(tensors)
        if len(tensors) != length:
            raise ValueError(f"{name} has {len(tensors)} tensors, params {length}")
        # (one pass by type where all is right; an entry of master may be None)
        if not _tensor_types(name == "master").issuperset(map(type, tensors)):
            tensor = _env().torch.Tensor
            for i, t in enumerate(tensors):
                if not isinstance(t, tensor) and not (name == "master" and t is None):
                    raise ValueError(f"{name}[{i}] must be a tensor, not {t!r}")


@lru_cache(maxsize=64)
def _words(count):
    return struct.Struct(f"{count}q")


def _column(c, name, tensors, shapes, dtype):
    """Pointers of a list of contiguous tensors (dtype None: of any).  A step of many small tensors is bound by the
    host: what is right costs a few passes over the list, and only what is not is looked at tensor by tensor."""
    tensor = c.env.torch.Tensor
    if (set(map(tensor.get_device, tensors)) != {c.index} or not all(map(tensor.is_contiguous, tensors))
            or (dtype is not None and set(map(_dtype_of, tensors)) != {dtype}) or list(map(_shape_of, tensors)) != shapes
            or c.other is not None or (any(map(_tracked, tensors)) and c.env.grad_enabled())):
        return [c.plain(name, t, shape, dtype or t.dtype) for t, shape in zip(tensors, shapes)]
    return list(map(tensor.data_ptr, tensors))


def adamw_step(params, grads, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, master=None,
               m_scale=None, v_scale=None, grad_scale=1.0, seed=0, stream=None):
    """One step of AdamW with decoupled weight decay on lists of contiguous tensors:
    params bf16, fp16 or fp32; grads of the same dtype or fp32; m and v fp32, or float8_e4m3fn and float8_e5m2 with
    m_scale and v_scale (adamw_states).  master, for params in 16 bits: their values in fp32, which the step updates
    and params then are the rounding of; an entry may be None.  step counts from 1.  Gradients are multiplied by
    grad_scale first (clipping, loss scales).  8-bit states round at random, by numbers that follow from seed, step
    and each value's place in the lists: calls of one step (groups of parameters) draw the same numbers unless each has a
    seed of its own.  step (int32), lr and grad_scale (fp32) may be tensors of one value on the device: a
    captured call then reads them at each replay."""
    _lists(params=params, grads=grads, m=m, v=v, master=master, m_scale=m_scale, v_scale=v_scale)
    if (m_scale is None) != (v_scale is None):
        raise ValueError("m_scale and v_scale come together")
    if not params:
        return
    codes = m_scale is not None
    count = len(params)
    n = _lib.MoeAdamw(0.0, betas[0], betas[1], eps, weight_decay, 1.0, int(seed) & 0xFFFFFFFFFFFFFFFF, 0,
                      8 if codes else 32, None, None, None)
    with _Call(params[0], stream) as c:
        env = c.env
        float32, plain = env.float32, c.plain
        m_type, v_type = (env.e4m3, env.e5m2) if codes else (float32, float32)

        def number(name, value, dtype):
            """A number, or the pointer of one on the device."""
            if isinstance(value, env.torch.Tensor):
                if value.numel() != 1:
                    raise ValueError(f"{name} must be one value, not {list(value.shape)}")
                return 0, plain(name, value, value.shape, dtype)
            return value, None

        n.lr, n.device_lr = number("lr", lr, float32)
        n.grad_scale, n.device_grad_scale = number("grad_scale", grad_scale, float32)
        step, n.device_step = number("step", step, env.int32)
        step = index(step)
        if not 0 <= step < 1 << 31:
            raise ValueError(f"step={step} is out of range")
        n.step = step
        shapes = list(map(_shape_of, params))
        pointers = [_column(c, "params", params, shapes, None), _column(c, "grads", grads, shapes, None)]
        if master is None:
            pointers.append([0] * count)
            wide = ()
        else:
            given = [i for i in range(count) if master[i] is not None]
            wide = [master[i] for i in given]
            pointers.append([0] * count)
            for i, at in zip(given, _column(c, "master", wide, [shapes[i] for i in given], float32)):
                pointers[2][i] = at
        pointers += [_column(c, "m", m, shapes, m_type), _column(c, "v", v, shapes, v_type)]
        values = list(map(env.torch.Tensor.numel, params))
        if codes:
            blocks = [((x + 127) // BLOCK,) for x in values]
            pointers += [_column(c, "m_scale", m_scale, blocks, float32), _column(c, "v_scale", v_scale, blocks, float32)]
        else:
            pointers += [[0] * count] * 2
        types = {t: _type(t) for t in set(map(_dtype_of, params)) | set(map(_dtype_of, grads))}
        kinds = [types[p.dtype] | types[g.dtype] << 32 for p, g in zip(params, grads)]
        # the C structs (7 pointers, the count, two 32-bit types) as 64-bit words: setting their fields one by one
        # would take longer than the checks
        table = _words(9 * count).pack(*chain.from_iterable(zip(*pointers, values, kinds)))
        _lib.check(c.lib.moe_adamw_step(ctypes.byref(n), count, table, c.stream))
    env.overwritten([*params, *wide, *m, *v, *(m_scale or ()), *(v_scale or ())])
