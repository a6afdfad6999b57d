"""AdamW's random numbers and refusals: which value draws which number, on both
sides of 2^32 values and from call to call, and lists with something other than
tensors in them."""

import numpy as np
import pytest

from gpu_util import require_gpu, say
from test_gpu_adamw import F32, HYPER, M_CODE, MASK, V_CODE, Step, coded, compare, mix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


def draws_from(seed, step, tensor, first, count):
    """The numbers of values first .. first + count - 1 of a tensor."""
    key = np.uint64(seed) & MASK
    for part in (seed >> 32, step, tensor):
        key = mix(part, key)
    value = np.arange(first, first + count, dtype=np.uint64)
    high = value >> np.uint64(32)
    out = np.empty(count, np.uint64)
    for h in np.unique(high):
        out[high == h] = mix(value[high == h], mix(h, key))
    return out


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad,master", [("float32", "float32", False), ("bfloat16", "bfloat16", True),
                                               ("float16", "float32", False)])
def test_around_a_thread_blocks_values(torch, moe, dtype, grad, master, bits):
    """A block of threads takes 2048 values."""
    shapes = [(2047,), (2048,), (2049,), (2048 + 127,), (2 * 2048 - 1,), (3 * 2048 + 1,), (16 * 2048,)]
    s = Step(torch, shapes, getattr(torch, dtype), getattr(torch, grad), bits, master)
    for step, seed in ((1, 3), (2, (5 << 32) + 1)):
        expected = s.expected(step, seed=seed, **HYPER)
        moe.adamw_step(step=step, seed=seed, **s.kwargs(), **HYPER)
        compare(torch, s, expected)


def test_codes_on_both_sides_of_32_bits(torch, moe):
    """Codes and scales to the last bit: of the first values, of those before 2^32 and of those behind it, which have the
    first ones' gradients and draw numbers of their own."""
    say("adamw past 2^32 values")
    far, seed = 1 << 32, (3 << 32) + 17
    n = far + 1000
    spans = [(0, 1000), (far - 2560, 2560 + 1000)]  # whole blocks of 128, but for the last
    gen = torch.Generator(device="cuda").manual_seed(4)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    states = moe.adamw_states([p], bits=8)
    for step in (1, 2):
        for at, count in spans:
            g[at:at + count] = torch.randn(count, generator=gen, device="cuda").bfloat16()
        g[far:] = g[:1000]
        expected = []
        for at, count in spans:
            where = slice(at, at + count)
            blocks = slice(at // 128, (at + count + 127) // 128)
            grad = g[where].float().cpu().numpy()

            def old(name):
                scale = np.repeat(states[name + "_scale"][0][blocks].cpu().numpy(), 128)[:count]
                return states[name][0][where].float().cpu().numpy() * scale

            b1, b2 = HYPER["betas"]
            m = old("m") * F32(b1) + grad * F32(1 - b1)
            v = old("v") * F32(b2) + (grad * grad) * F32(1 - b2)
            u = draws_from(seed, step, 0, at, count)
            expected.append((where, blocks, coded(m, u & np.uint64(0xFFFF), *M_CODE), coded(v, u >> np.uint64(16), *V_CODE)))
        moe.adamw_step([p], [g], step=step, seed=seed, **states, **HYPER)
        for where, blocks, m, v in expected:
            for name, (value, scale) in (("m", m), ("v", v)):
                assert np.array_equal(states[name][0][where].float().cpu().numpy(), value), (where, name, step)
                assert np.array_equal(states[name + "_scale"][0][blocks].cpu().numpy(), scale), (where, name, step)
        first, behind = states["m"][0][:896].view(torch.uint8), states["m"][0][far:far + 896].view(torch.uint8)
        assert (first != behind).any()


def test_a_number_follows_from_the_place_in_the_call(torch, moe):
    """A tensor alone in a call draws what the first of several does: calls of one step take seeds of their own."""
    def one():
        s = Step(torch, [(5000,)], torch.bfloat16, torch.bfloat16, 8, False)
        return s

    def codes(s):
        return s.m[0].view(torch.uint8).clone()

    a, b, c = one(), one(), one()
    moe.adamw_step(step=1, seed=8, **a.kwargs())
    moe.adamw_step(step=1, seed=8, **b.kwargs())
    moe.adamw_step(step=1, seed=9, **c.kwargs())
    assert torch.equal(codes(a), codes(b)) and not torch.equal(codes(a), codes(c))
    pair = [one(), one()]
    together = {name: x + y for (name, x), y in zip(pair[0].kwargs().items(), pair[1].kwargs().values())}
    moe.adamw_step(step=1, seed=8, **together)
    assert torch.equal(codes(pair[0]), codes(a)) and not torch.equal(codes(pair[1]), codes(a))


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_no_tensor_is_named(torch, moe, bits):
    s = Step(torch, [(300,), (64,)], torch.bfloat16, torch.bfloat16, bits, True)
    before = s.state()
    for name, tensors in s.kwargs().items():
        for at in (0, 1):
            for bad in ((1.0, "x") if name == "master" else (None, 1.0)):
                some = list(tensors)
                some[at] = bad
                with pytest.raises(ValueError, match=rf"{name}\[{at}\] must be a tensor"):
                    moe.adamw_step(**{**dict(step=1), **s.kwargs(), name: some})
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s.state(), before))
