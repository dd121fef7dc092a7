"""GPU checks of scored routing and its gradient at the edges of their number formats, against the
float64 forms of ref64."""
import numpy as np
import pytest
import torch

import indirect_expert_matmul_amd as moe
import ref64
from moe_testutil import dev_f32, dev_i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_group_sums_past_float32(score, dtype):
    """Biases of the lowest float32 as a mask: the sum of two of them is no float32, but it ranks its
    group above groups without an expert, and sums past the range above 0 rank by their size."""
    low = np.finfo(np.float32).min
    l = torch.from_numpy(np.random.default_rng(1).standard_normal((37, 16))).to(dtype)
    b = np.full(16, -np.inf)                 # groups of 4
    b[4:8] = low
    b[8:12] = np.linspace(-0.1, 0.1, 4)
    up = np.zeros(16)
    up[0:4], up[4:8], up[12:16] = -low / 1.5, -low / 1.25, -low
    down = np.array([low / 1.25] * 4 + [low] * 4 + [low / 1.5] * 4 + [low / 1.75] * 4)
    for bias, keep, k in ((b, 2, 6), (b, 3, 9), (up, 1, 3), (up, 2, 7), (down, 1, 2), (down, 3, 12)):
        kw = dict(score=score, n_group=4, topk_group=keep)
        ids, w = moe.moe_router_scored(l.cuda(), k, bias=dev_f32(bias), **kw)
        ri, _, _ = ref64.route(l.double().numpy(), k, bias=np.float32(bias), **kw)
        assert np.array_equal(ids.cpu().numpy(), ri), (keep, k)
