"""Differential attention at the borders of its values: scores of -inf, queries
without a value, large values, one weight that holds a row, and gradients at
q, k, v decoded from 8 bits.  The bounds are those of test_gpu_diff's docstring
where nothing else is said."""
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl
from test_gpu_diff import check_forward, decode_reference, make, maps, reference_gradients, rows_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("late", [150, 158, 199])
def test_one_weight_that_holds_a_row_is_exact(late, d):
    """A late key that outweighs all the others gives its own value: the weight and the sum that it is divided by are
    rounded alike, whatever the weight is.

    Key 0 has the level 0, key `late` a level of L = 12.4 to 15.5 (in log2, by row) and all the others -86, so the rest of
    the row weighs 2^-12.4 of it at most.  With |v| in [1, 2), values 4 apart at most, it moves the output by 2^-10.4, and
    a bf16 value of 1 or more is left by 2^-9 at least."""
    N = 200
    keep = np.ones((1, 2, 2), bool)
    q, k, v, _, _, rp, ci, *_ = make(1, N, 1, d, keep, 43)
    level = 12.5 + 3 * torch.arange(N, device="cuda") / N
    q.zero_()
    k.zero_()
    for m in (0, d // 2):
        q[0, :, 0, m] = (level * math.log(2.0)).bfloat16()
        q[0, :, 0, m + 1] = 60.0
        k[0, :, 0, m + 1] = -1.0
        k[0, 0, 0, m + 1] = k[0, late, 0, m + 1] = 0
        k[0, late, 0, m] = 1
    v = ((1 + torch.rand(v.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(44)) * 0.99)
         * torch.where(torch.rand(v.shape, device="cuda") < 0.5, -1.0, 1.0)).bfloat16().clamp(-1.9921875, 1.9921875)
    want = v[:, late:late + 1].expand(1, N, 1, d)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, torch.zeros(1, device="cuda"), softmax_scale=1.0)
    assert torch.equal(out, want) and torch.equal(out2, want)
    assert torch.equal(out, sl.diff_attn_forward(q, k, v, rp, ci, torch.zeros(1, device="cuda"), softmax_scale=1.0))
