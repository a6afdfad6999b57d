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

from . import _lib
from .products import _Call, _type

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


def adamw_step(params, grads, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, master=None,
               m_scale=None, v_scale=None, grad_scale=1.0, seed=0, stream=None):
    """One step of AdamW with decoupled weight decay on lists of contiguous tensors:
    params bf16, fp16 or fp32; grads of the same dtype or fp32; m and v fp32, or float8_e4m3fn and float8_e5m2 with
    m_scale and v_scale (adamw_states).  master, for params in 16 bits: their values in fp32, which the step updates
    and params then are the rounding of; an entry may be None.  step counts from 1.  Gradients are multiplied by
    grad_scale first (clipping, loss scales).  8-bit states round at random, by numbers that follow from seed, step
    and each value's place.  step (int32), lr and grad_scale (fp32) may be tensors of one value on the device: a
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
        float32, types, plain = env.float32, env.types, c.plain
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
        if not 0 <= int(step) < 1 << 31:
            raise ValueError(f"step={step} is out of range")
        n.step = int(step)
        # the C structs (7 pointers, the count, two 32-bit types) as 64-bit words: setting their fields one by one
        # would take longer than the checks
        table = []
        wide = ms = vs = 0
        for i in range(count):
            p, g = params[i], grads[i]
            shape, dtype = p.shape, p.dtype
            values = p.numel()
            if master is not None:
                wide = 0 if master[i] is None else plain("master", master[i], shape, float32)
            if codes:
                blocks = ((values + 127) // BLOCK,)
                ms = plain("m_scale", m_scale[i], blocks, float32)
                vs = plain("v_scale", v_scale[i], blocks, float32)
            table += (plain("params", p, shape, dtype), plain("grads", g, shape, g.dtype), wide,
                      plain("m", m[i], shape, m_type), plain("v", v[i], shape, v_type), ms, vs, values,
                      (types[dtype] if dtype in types else _type(dtype))
                      | (types[g.dtype] if g.dtype in types else _type(g.dtype)) << 32)
        words = (ctypes.c_int64 * len(table))(*table)
        _lib.check(c.lib.moe_adamw_step(ctypes.byref(n), count,
                                        ctypes.cast(words, ctypes.POINTER(_lib.MoeAdamwTensor)), c.stream))
    env.torch.autograd.graph.increment_version(params)
