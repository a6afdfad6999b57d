"""Autograd's version counters: a call raises that of every tensor that it
overwrites, so that a backward pass through what stood there before is refused,
and of no other."""

import pytest

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def moe(torch):
    import expert_ffn_layer_router_amd as m
    return m


def raised(call, tensors):
    """Whether the call raised each tensor's version."""
    before = [t._version for t in tensors]
    call()
    return [t._version > b for t, b in zip(tensors, before)]


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_raises_what_it_writes(torch, moe, bits):
    params = [torch.ones(40, device="cuda").bfloat16(), torch.ones(7, device="cuda")]
    grads = [torch.ones_like(p) for p in params]
    master = [params[0].float(), None]
    states = moe.adamw_states(params, bits=bits)
    written = params + master[:1] + [t for tensors in states.values() for t in tensors]
    lr = torch.tensor(1e-3, device="cuda")
    assert all(raised(lambda: moe.adamw_step(params, grads, step=1, lr=lr, master=master, **states), written))
    assert not any(raised(lambda: moe.adamw_step(params, grads, step=2, lr=lr, master=master, **states), grads + [lr]))


def test_backward_through_a_masters_old_values_is_refused(torch, moe):
    """The usual leaf where 16-bit weights are the rounding of 32-bit ones."""
    master = torch.ones(128, device="cuda", requires_grad=True)
    loss = (master * master).sum()
    param = master.detach().bfloat16()
    states = moe.adamw_states([param])
    with torch.no_grad():
        moe.adamw_step([param], [torch.ones_like(param)], step=1, master=[master], **states)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_have_no_version(torch, moe):
    with torch.inference_mode():
        param = torch.ones(128, device="cuda").bfloat16()
        states = moe.adamw_states([param], bits=8)
        master = param.float()
        moe.adamw_step([param], [torch.ones_like(param)], step=1, lr=0.1, master=[master], **states)
        assert torch.equal(param, master.bfloat16()) and (param < 1).all()
