"""Infinities of the open page in a request that many CTAs share, where a token far back has nearly
all of the weight: the rows that attend them are infinite, as where one CTA has the request alone."""
import math

import pytest
import torch

from tests.test_gpu_paged import BF16, F16
from tests.test_gpu_paged_attend import Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16), (128, F16)])
@pytest.mark.parametrize("n,m", [(20000, 5), (9000, 300), (300, 3)])
@pytest.mark.parametrize("lead", [20.0, 300.0, 5000.0])
def test_infinities_beside_a_large_weight_far_back(d, dtype, n, m, lead):
    """`lead`: by how much (as a power of 2) the early token's weight is the largest."""
    f = Filled([n + 7], [m], 4, 2, d, 32, "int8", dtype, seed=2)
    n += 7
    c, row = f.cache, n % 32 - 3
    assert row > 0
    c.pages(0)[f.table[0, 0].item(), :, 0, 0] = 0
    c.pages(0)[f.table[0, 0].item(), :, 0, 0, 0] = 100
    c.pages(0)[f.table[0, 0].item(), :, 0, 1:] = 0
    c.scales(0)[f.table[0, 0].item(), :, 0] = lead * math.log(2.0) / 100
    c.scales(0)[f.table[0, 1:(n // 32)].long(), :, 0] *= 2.0 ** -10
    c.tails(0)[:, :, 0] *= 2.0 ** -10
    q = f.q.clone()
    q[..., 0] = 1
    for value in (math.inf, -math.inf, math.nan):
        c.tails(0)[0, 1, 1, row, 5] = 0.0
        want = f.attend(q=q, scale=1.0)
        c.tails(0)[0, 1, 1, row, 5] = value
        first = n // 32 * 32 + row - (n - m)  # the token at that position
        want[max(first, 0):, 2:, 5] += value
        out = f.attend(q=q, scale=1.0)
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out[~out.isnan()], want[~want.isnan()])
    # both kinds at once
    c.tails(0)[0, 1, 1, row - 1, 5], c.tails(0)[0, 1, 1, row, 5] = math.inf, -math.inf
    out = f.attend(q=q, scale=1.0)
    assert out[-1, 2:, 5].isnan().all() and c.status() == 0
