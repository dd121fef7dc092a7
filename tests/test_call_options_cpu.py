"""The option structs that the binding makes once per set of values are made per value, never per object."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe


@pytest.mark.parametrize("make", [lambda v: torch.tensor(v), lambda v: np.array(v), lambda v: np.array(v)[()],
                                  float])
def test_numbers_that_change_in_place(make):
    """A 0-d tensor or array as scale or tau: its value at the call counts, not the one of an earlier call."""
    s = make(1.0)
    assert moe._router_config("sigmoid", 1, 1, 1, True, s).scale == 1.0
    assert moe._call_options(0, s, None, 0).tau == 1.0
    if isinstance(s, (torch.Tensor, np.ndarray)):
        s[...] = 2.5
        assert moe._router_config("sigmoid", 1, 1, 1, True, s).scale == 2.5
        assert moe._call_options(0, s, None, 0).tau == 2.5


def test_whole_numbers_of_other_types():
    n = torch.tensor(2)
    c = moe._router_config("softmax", n, n, np.int32(1), np.bool_(False), 1)
    assert (c.n_group, c.topk_group, c.group_top, c.renorm) == (2, 2, 1, 0)
    n += 2
    c = moe._router_config("softmax", n, n, 1, torch.tensor(True), 1)
    assert (c.n_group, c.topk_group, c.renorm) == (4, 4, 1)
    p = torch.tensor(1)
    assert moe._call_options(p, 0.0, None, p).path == 1
    p += 1
    o = moe._call_options(p, 0.0, None, p)
    assert (o.path, o.act_quant) == (2, 2)
    for bad in (dict(score="tanh"), dict(n_group=1.5), dict(scale="x")):
        kw = dict(dict(score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0), **bad)
        with pytest.raises((ValueError, TypeError)):
            moe._router_config(**kw)


def test_same_values_same_struct():
    a = moe._router_config("sigmoid", 8, 4, 2, True, 2.5)
    assert moe._router_config("sigmoid", 8, 4, 2, True, 2.5) is a
    assert moe._call_options(1, 0.0, None, 2) is moe._call_options(1, 0.0, None, 2)
