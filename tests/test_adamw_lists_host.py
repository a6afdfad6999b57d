"""Host-only test of the lists that adamw_step takes: an entry that is no tensor
(a parameter without a gradient has None) is refused by its name and place,
before any device is looked at."""

import pytest


def test_what_is_no_tensor_is_named():
    import torch

    import expert_ffn_layer_router_amd as moe

    class Own(torch.Tensor):
        """A subclass is a tensor too."""

    x = [torch.zeros(4), torch.nn.Parameter(torch.zeros(3)), torch.zeros(2).as_subclass(Own)]
    lists = dict(params=x, grads=x, m=x, v=x, master=[None, x[1], x[2]], m_scale=x, v_scale=x)
    for name, tensors in lists.items():
        for at in range(3):
            for bad in (None, 1.0, "x", tensors):
                if name == "master" and bad is None:
                    continue
                some = list(tensors)
                some[at] = bad
                with pytest.raises(ValueError, match=rf"^{name}\[{at}\] must be a tensor"):
                    moe.adamw_step(**{**lists, name: some}, step=1)
    with pytest.raises(ValueError, match="on a GPU"):  # what is right goes on to the device
        moe.adamw_step(**lists, step=1)
