"""AdamW on the GPU.

m and v before their rounding, their scales and their codes are fp32 operations
in a given order (moe_optim.h), each rounded to nearest: numpy's fp32 ones give
the same bits.  The weights are compared with 64 bits; e = 2^-24:
  m, v     three roundings each (a product of each term, their sum), the
           gradient's scaling one more: 4e of |beta m| + |(1 - beta) g|; of v
           6e of itself
  update   rate m / (sqrt(v) root + eps): m's error, v's at most 3e through the
           root, and 8 operations of e (the root, the division and the
           reciprocal may be off by 2e): 20e of |rate m / (..)| where m's terms
           do not cancel, 4e (|beta m| + |(1 - beta) g|) rate / (..) more
  weights  the decay's product and the difference: 3e |p|, then the output's
           rounding
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
F32 = np.float32
MASK = np.uint64(0xFFFFFFFF)


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


def fold(x, c):
    p = (np.asarray(x, np.uint64) & MASK) * np.uint64(c)
    return ((p >> np.uint64(32)) ^ p) & MASK


def mix(x, key):
    key = np.uint64(key)
    return fold((fold(np.asarray(x, np.uint64) ^ key, 0x9E3779B9) + key) & MASK, 0xBB67AE85)


def draws(seed, step, tensor, count):
    key = np.uint64(seed) & MASK
    for part in (seed >> 32, step, tensor, 0):
        key = mix(part, key)
    return mix(np.arange(count, dtype=np.uint64), key)


def coded(x, u, most, lowest, bits):
    """(codes' values, scales) of fp32 x with the random numbers u of 16 bits."""
    blocks = -(-x.size // 128)
    whole = np.zeros(blocks * 128, F32)
    whole[:x.size] = x
    rand = np.zeros(blocks * 128, F32)
    rand[:x.size] = u.astype(F32) / F32(65536)
    whole, rand = whole.reshape(blocks, 128), rand.reshape(blocks, 128)
    top = np.abs(whole).max(1, keepdims=True)
    scale = top * (F32(1) / F32(most))
    y = np.abs(whole) / np.where(scale > 0, scale, F32(1))
    unit = np.maximum(np.frexp(y)[1] - 1, lowest) - bits
    n = np.floor(np.ldexp(y, -unit) + rand)
    if bits == 2:
        n = np.where((n == 0) & (whole > 0), F32(1), n)
    value = np.copysign(np.minimum(np.ldexp(n, unit), F32(most)), whole)
    return value.reshape(-1)[:x.size], scale[:, 0]


M_CODE, V_CODE = (448.0, -6, 3), (57344.0, -14, 2)


class Step:
    """Tensors of the given shapes and what a step makes of them."""

    def __init__(self, torch, shapes, dtype, grad, bits, master, seed=0, moments=True):
        gen = torch.Generator().manual_seed(seed)
        self.torch, self.bits = torch, bits

        def normal(shape, std):
            return torch.randn(shape, generator=gen) * std

        self.params, self.grads, self.master, self.m, self.v, self.m_scale, self.v_scale = [], [], [], [], [], [], []
        for s in shapes:
            wide = normal(s, 0.1)
            self.params.append(wide.to(dtype).cuda())
            self.master.append(wide.cuda() if master else None)
            self.grads.append((normal(s, 1e-2) * torch.exp(normal(s, 1))).to(grad).cuda())
            m, v = normal(s, 1e-2), normal(s, 1e-2) ** 2
            if not moments:
                m, v = m * 0, v * 0
            if bits == 8:
                half = np.full(m.numel(), 32768, np.uint64)
                for x, code, kind, to, scales in ((m, M_CODE, torch.float8_e4m3fn, self.m, self.m_scale),
                                                  (v, V_CODE, torch.float8_e5m2, self.v, self.v_scale)):
                    c, sc = coded(x.numpy().reshape(-1), half, *code)
                    to.append(torch.from_numpy(c).view(s).to(kind).cuda())
                    scales.append(torch.from_numpy(sc).cuda())
            else:
                self.m.append(m.cuda())
                self.v.append(v.cuda())

    def kwargs(self):
        d = dict(params=self.params, grads=self.grads, m=self.m, v=self.v)
        if any(x is not None for x in self.master):
            d["master"] = self.master
        if self.bits == 8:
            d.update(m_scale=self.m_scale, v_scale=self.v_scale)
        return d

    def state(self):
        out = []
        for name in ("params", "master", "m", "v", "m_scale", "v_scale"):
            out += [x.clone() for x in getattr(self, name) if x is not None]
        return out

    def expected(self, step, lr, betas, eps, weight_decay, grad_scale=1.0, seed=0):
        """A list of (params in 64 bits, bound before rounding, m, v, m_scale, v_scale) on the host."""
        b1, b2 = betas
        out = []
        for i, p in enumerate(self.params):
            g = self.grads[i].float().cpu().numpy().reshape(-1) * F32(grad_scale)
            m, v = (x[i].float().cpu().numpy().reshape(-1) for x in (self.m, self.v))
            if self.bits == 8:
                spread = lambda s: np.repeat(s[i].cpu().numpy(), 128)[:m.size]  # noqa: E731
                m, v = m * spread(self.m_scale), v * spread(self.v_scale)
            terms = np.abs(b1 * m.astype(np.float64)) + np.abs((1 - b1) * g.astype(np.float64))
            m1 = m * F32(b1) + g * F32(1 - b1)
            v1 = v * F32(b2) + (g * g) * F32(1 - b2)
            w = (self.master[i] if self.master[i] is not None else p).double().cpu().numpy().reshape(-1)
            m64 = b1 * m.astype(np.float64) + (1 - b1) * g.astype(np.float64)
            v64 = b2 * v.astype(np.float64) + (1 - b2) * g.astype(np.float64) ** 2
            per = lr / (1 - b1 ** step) / (np.sqrt(v64) / np.sqrt(1 - b2 ** step) + eps)
            new = w * (1 - lr * weight_decay) - per * m64
            off = 3 * E * np.abs(w) + 20 * E * np.abs(per * m64) + 4 * E * terms * per + E * np.abs(new)
            sm = sv = None
            if self.bits == 8:
                u = draws(seed, step, i, m.size)
                m1, sm = coded(m1, u & np.uint64(0xFFFF), *M_CODE)
                v1, sv = coded(v1, u >> np.uint64(16), *V_CODE)
            out.append((new, off, m1, v1, sm, sv))
        return out


def compare(torch, s, expected):
    for i, (new, off, m, v, sm, sv) in enumerate(expected):
        p = s.params[i]
        got = p.double().cpu().numpy().reshape(-1)
        half = torch.finfo(p.dtype).eps / 2
        floor = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[p.dtype]
        bound = off + half * (np.abs(new) + off) + floor
        assert (np.abs(got - new) <= bound).all(), (i, np.abs(got - new).max())
        if s.master[i] is not None:
            wide = s.master[i].double().cpu().numpy().reshape(-1)
            assert (np.abs(wide - new) <= off + E * np.abs(new)).all(), i
            assert torch.equal(s.master[i].to(p.dtype), p)
        assert np.array_equal(s.m[i].float().cpu().numpy().reshape(-1), m), i
        assert np.array_equal(s.v[i].float().cpu().numpy().reshape(-1), v), i
        if s.bits == 8:
            assert np.array_equal(s.m_scale[i].cpu().numpy(), sm), i
            assert np.array_equal(s.v_scale[i].cpu().numpy(), sv), i


HYPER = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
# every remainder of 8 and of 128, one value, none, and more than a block's 4096 values
SHAPES = [(1,), (7,), (8,), (9,), (127,), (128,), (129,), (0,), (3, 5, 7), (4095,), (4096,), (4097,), (65, 321), (12345,)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad,master", [("float32", "float32", False), ("bfloat16", "bfloat16", False),
                                               ("bfloat16", "float32", True), ("float16", "float16", True),
                                               ("float16", "float32", False), ("bfloat16", "bfloat16", True)])
def test_adamw(torch, moe, dtype, grad, master, bits):
    say(f"adamw {dtype} {grad} {master} {bits}")
    s = Step(torch, SHAPES, getattr(torch, dtype), getattr(torch, grad), bits, master)
    for step, seed in ((1, 0), (2, 5), (1000, (7 << 32) + 9)):
        expected = s.expected(step, seed=seed, **HYPER)
        moe.adamw_step(step=step, seed=seed, **s.kwargs(), **HYPER)
        compare(torch, s, expected)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(torch, moe, bits):
    """More tensors than a launch takes, of all types in turn."""
    kinds = [("float32", "float32", False), ("bfloat16", "bfloat16", True), ("float16", "float32", False)]
    parts = [Step(torch, [(17 * i + 1,) for i in range(40)], getattr(torch, d), getattr(torch, g), bits, m, seed=n)
             for n, (d, g, m) in enumerate(kinds)]
    s = parts[0]
    for name in ("params", "grads", "master", "m", "v", "m_scale", "v_scale"):
        lists = [getattr(p, name) for p in parts]
        setattr(s, name, [x for group in zip(*lists) for x in group])
    expected = s.expected(3, seed=11, **HYPER)
    moe.adamw_step(step=3, seed=11, **s.kwargs(), **HYPER)
    compare(torch, s, expected)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-8, 1.0, 1e4])
def test_any_eps(torch, moe, eps, bits):
    """Gradients of 2^-62 to 2^4, whose v is subnormal below 2^-58: it is off by 2^-150 more, half of that through the
    root."""
    say(f"adamw eps {eps} {bits}")
    s = Step(torch, [(1000,), (131,)], torch.float32, torch.float32, bits, False, moments=False)
    gen = torch.Generator().manual_seed(3)
    for g in s.grads:
        g.copy_(torch.sign(torch.randn(g.shape, generator=gen)) * 2 ** (torch.rand(g.shape, generator=gen) * 66 - 62))
    hyper = dict(HYPER, eps=eps)
    expected = []
    for g, (new, off, *rest) in zip(s.grads, s.expected(1, **hyper)):
        g64 = g.double().cpu().numpy()
        per = hyper["lr"] / (np.abs(g64) + eps) * np.abs(g64)
        expected.append((new, off + per * 2.0 ** -151 / (1e-3 * g64 ** 2), *rest))
    assert min(g.abs().min().item() for g in s.grads) < 2.0 ** -60
    moe.adamw_step(step=1, **s.kwargs(), **hyper)
    compare(torch, s, expected)


def test_first_step_from_zero_states(torch, moe):
    for bits in (8, 32):
        s = Step(torch, [(300,), (2, 64)], torch.bfloat16, torch.float32, bits, True, moments=False)
        states = moe.adamw_states(s.params, bits=bits)
        for name, tensors in states.items():
            assert [(t.shape, t.dtype) for t in tensors] == [(t.shape, t.dtype) for t in getattr(s, name)]
            setattr(s, name, tensors)
        expected = s.expected(1, **HYPER)
        moe.adamw_step(s.params, s.grads, step=1, master=s.master, **states, **HYPER)
        compare(torch, s, expected)


def test_against_torch(torch, moe):
    s = Step(torch, [(64, 33), (5,)], torch.float32, torch.float32, 32, False, moments=False)
    ref = [torch.nn.Parameter(p.double()) for p in s.params]
    opt = torch.optim.AdamW(ref, **HYPER)
    for step in range(1, 6):
        for r, g in zip(ref, s.grads):
            r.grad = g.double() * step
        opt.step()
        moe.adamw_step(s.params, [g * step for g in s.grads], s.m, s.v, step, **HYPER)
    for r, p in zip(ref, s.params):
        # five steps of the bound above; an update is below 2 lr here
        assert ((r.detach() - p.double()).abs() <= 5 * E * (5 * r.detach().abs() + 40 * 2 * HYPER["lr"])).all()


def test_8_bit_states_keep_their_mean(torch, moe):
    """With one gradient over many steps v moves by a thousandth of itself at a time, a hundred times less than its
    codes are apart: the mean over many values follows all the same."""
    n = 1 << 16
    p = torch.zeros(n, device="cuda")
    g = torch.ones(n, device="cuda")
    states = moe.adamw_states([p], bits=8)
    steps = 600
    for step in range(1, steps + 1):
        moe.adamw_step([p], [g], step=step, lr=0.0, seed=3, **states)
    v = states["v"][0].double() * states["v_scale"][0].double().repeat_interleave(128)
    m = states["m"][0].double() * states["m_scale"][0].double().repeat_interleave(128)
    # A step's rounding moves a value by less than a quarter of itself (e5m2), with mean zero; what is left of it decays
    # by 0.999 a step.  The variance that a step adds is at most frac (1 - frac) / 16 of the value's square, frac at
    # most 0.001 x 8 while v is near its mean: the sum over steps below 600 x 0.008 / 16 = 0.3, so the mean of n
    # values is off by less than 6 x sqrt(0.3 / n) = 1.3% (six standard deviations)
    assert abs(v.mean().item() / (1 - 0.999 ** steps) - 1) < 0.013
    assert abs(m.mean().item() - 1) < 0.013


def test_numbers_on_the_device(torch, moe):
    a = Step(torch, [(1000,), (33, 7)], torch.bfloat16, torch.bfloat16, 8, True)
    b = Step(torch, [(1000,), (33, 7)], torch.bfloat16, torch.bfloat16, 8, True)
    lr, scale = torch.tensor([3e-3], device="cuda"), torch.tensor(0.5, device="cuda")
    step = torch.tensor([7], dtype=torch.int32, device="cuda")
    moe.adamw_step(step=7, lr=float(lr.item()), grad_scale=0.5, seed=1, **a.kwargs())
    moe.adamw_step(step=step, lr=lr, grad_scale=scale, seed=1, **b.kwargs())
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.state(), b.state()))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays(torch, moe, bits):
    """A captured step with its numbers on the device, replayed with others and with eager work between."""
    a = Step(torch, [(5000,), (129,)], torch.bfloat16, torch.float32, bits, True)
    b = Step(torch, [(5000,), (129,)], torch.bfloat16, torch.float32, bits, True)
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda")
    before = [x.clone() for x in a.state()]
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            moe.adamw_step(step=step, lr=lr, **a.kwargs())
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.state(), before))
    for t, rate in ((1, 1e-3), (2, 5e-4), (3, 2e-3), (4, 1e-3)):
        step.fill_(t)
        lr.fill_(rate)
        for g in a.grads + b.grads:
            g.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        moe.adamw_step(step=t, lr=float(torch.tensor(rate).item()), **b.kwargs())
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.state(), b.state()))


def test_nonfinite_gradients_stay_in_their_block(torch, moe):
    for bits in (32, 8):
        s = Step(torch, [(1024,)], torch.bfloat16, torch.float32, bits, True)
        clean = Step(torch, [(1024,)], torch.bfloat16, torch.float32, bits, True)
        s.grads[0][200] = float("inf")
        s.grads[0][700] = float("nan")
        for step in (1, 2):
            moe.adamw_step(step=step, **s.kwargs(), **HYPER)
            moe.adamw_step(step=step, **clean.kwargs(), **HYPER)
        hit = torch.zeros(1024, dtype=torch.bool, device="cuda")
        if bits == 8:
            hit[128:256] = hit[640:768] = True
            assert s.m_scale[0][[1, 5]].isnan().all() and s.v_scale[0][[1, 5]].isnan().all()
        else:
            hit[200] = hit[700] = True
        for x, y in ((s.params[0], clean.params[0]), (s.m[0], clean.m[0]), (s.v[0], clean.v[0])):
            assert torch.equal(x.float()[~hit], y.float()[~hit])
        assert s.params[0][hit].isnan().all()


def test_streams_and_refusals(torch, moe):
    from expert_ffn_layer_router_amd import MoeError
    s = Step(torch, [(1000,), (64,)], torch.bfloat16, torch.bfloat16, 8, True)
    other = Step(torch, [(1000,), (64,)], torch.bfloat16, torch.bfloat16, 8, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    moe.adamw_step(step=1, stream=stream, **s.kwargs())
    torch.cuda.current_stream().wait_stream(stream)
    moe.adamw_step(step=1, **other.kwargs())
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s.state(), other.state()))
    before = s.state()

    def refused(error, **over):
        with pytest.raises(error):
            moe.adamw_step(**{**dict(step=1), **s.kwargs(), **over})

    refused(ValueError, grads=s.grads[:1])
    refused(ValueError, grads=[g.double() for g in s.grads])
    refused(ValueError, grads=[s.grads[0].cpu(), s.grads[1]])
    refused(ValueError, m=[x.float() for x in s.m])
    refused(ValueError, m_scale=None)
    refused(ValueError, m_scale=[x[1:] for x in s.m_scale])
    refused(ValueError, params=[torch.zeros(1000, 2, dtype=torch.bfloat16, device="cuda")[:, 0], s.params[1]])
    refused(ValueError, params=s.params[0])
    refused(ValueError, step=torch.tensor([1], device="cuda"))                   # 64 bits
    refused(ValueError, lr=torch.tensor([1.0, 2.0], device="cuda"))
    refused(ValueError, step=1 << 31)
    refused(TypeError, step=1.5)
    refused(MoeError, step=0)
    refused(MoeError, betas=(1.0, 0.9))
    refused(MoeError, lr=float("nan"))
    refused(MoeError, eps=-1.0)
    # the same tensor twice, and states that share memory
    refused(MoeError, params=[s.params[1], s.params[1]], grads=[s.grads[1]] * 2, master=[s.master[1]] * 2,
            m=[s.m[1]] * 2, v=[s.v[1]] * 2, m_scale=[s.m_scale[1]] * 2, v_scale=[s.v_scale[1]] * 2)
    refused(MoeError, m_scale=s.v_scale)
    refused(MoeError, grads=s.params)
    leaf = [p.clone().requires_grad_() for p in s.params]
    refused(ValueError, params=leaf)
    with torch.no_grad():
        moe.adamw_step(**{**dict(step=1), **other.kwargs(), "params": leaf})
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s.state(), before))
    moe.adamw_step([], [], [], [], 1)


def test_versions_views_and_scalars(torch, moe):
    """Autograd sees that a step overwrote its leaves; views need their alignment; a tensor may have no dimension."""
    from expert_ffn_layer_router_amd import MoeError
    p = torch.ones(4, device="cuda", requires_grad=True)
    y = (p * p).sum()
    states = moe.adamw_states([p])
    with torch.no_grad():
        moe.adamw_step([p], [torch.ones(4, device="cuda")], step=1, **states)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        q = torch.ones(4, device="cuda")
        moe.adamw_step([q], [torch.ones(4, device="cuda")], step=1, **moe.adamw_states([q]))
        assert torch.equal(q, p)
    one = [torch.tensor(1.0, device="cuda")]
    moe.adamw_step(one, [torch.tensor(1.0, device="cuda")], step=1, **moe.adamw_states(one))
    assert one[0].item() == p[0].item()
    buf = torch.ones(16, device="cuda")
    view = [buf[1:9]]
    with pytest.raises(MoeError, match="aligned"):
        moe.adamw_step(view, [torch.ones(8, device="cuda")], step=1, **moe.adamw_states(view))
    view = [buf[4:12]]
    moe.adamw_step(view, [torch.ones(8, device="cuda")], step=1, **moe.adamw_states(view))
    assert (buf[:4] == 1).all() and (buf[12:] == 1).all() and torch.equal(buf[4:8], p.detach())


def test_past_32_bits(torch, moe):
    """A tensor of more than 2^32 values: the last ones, and the first behind 2^32."""
    n = (1 << 32) + 1000
    tail = 5000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:] = torch.randn(tail, device="cuda").to(torch.bfloat16)
    g[-tail:] = torch.randn(tail, device="cuda").to(torch.bfloat16)
    old = p[-tail:].clone()
    states = moe.adamw_states([p], bits=8)
    moe.adamw_step([p], [g], step=1, seed=1, **states, **HYPER)
    # a first step: m = 0.1 g and v = 0.001 g^2 before their rounding, so each weight moves by lr against its gradient's sign
    w = old.double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * torch.sign(g[-tail:].double())
    assert ((p[-tail:].double() - w).abs() <= 2.0 ** -8 * w.abs() * 1.01 + 100 * E + 1e-3 * HYPER["lr"]).all()
    assert not p[:-tail].any() and not states["m"][0].view(torch.uint8)[:-tail].any()
    m = states["m"][0][-tail:].double() * states["m_scale"][0].repeat_interleave(128)[:n][-tail:].double()
    # an 8-bit state is one of its two neighbouring codes: within 2^-3 of itself, or 2^-9 of its scale
    top = states["m_scale"][0].repeat_interleave(128)[:n][-tail:].double()
    want = 0.1 * g[-tail:].double()
    assert ((m - want).abs() <= 2.0 ** -3 * want.abs() * 1.01 + 2.0 ** -9 * top * 1.01).all()
