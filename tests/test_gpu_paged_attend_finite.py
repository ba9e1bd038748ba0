"""Infinities and NaN in the open pages of many requests, chunk attention: each reaches the
rows from its token on, in its channel, and nothing else changes by a bit."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_paged import BF16, F16
from tests.test_gpu_paged_attend import Filled

pytestmark = pytest.mark.gpu


def steps(kind, r, rs):
    """Lengths and new tokens: blocks that both units share (more than 32 tokens at four heads a
    kv-head), blocks of one unit, and blocks of a single tile."""
    lens = rs.randint(1, {"tiles": 128, "mixed": 420, "long": 900}[kind], r)
    new = np.where(rs.uniform(size=r) < 0.5, rs.randint(1, 9, r), rs.randint(9, 150, r))
    return lens.tolist(), np.minimum(lens, new).tolist()


@pytest.mark.parametrize("kind,r", [("tiles", 500), ("mixed", 400), ("long", 200)])
@pytest.mark.parametrize("d,dtype,code", [(128, F16, "int8"), (128, BF16, "e4m3"), (64, F16, "e4m3"), (64, BF16, "int8")])
def test_marks_of_many_parts(kind, r, d, dtype, code):
    rs = np.random.RandomState(r + d)
    h, g, page = 8, 4, 64
    lens, new = steps(kind, r, rs)
    f = Filled(lens, new, h * g, h, d, page, code, dtype, seed=r)
    tails = f.cache.tails(0)
    # what is not finite: in half of the requests with open rows, in some of their heads, one or
    # two tokens each; past the length, where nothing may read, in all
    at, kinds = [], []
    for b in range(r):
        rows = lens[b] % page
        tails[b, :, :, rows:] = math.nan
        if rows and rs.uniform() < 0.5:
            for _ in range(rs.randint(1, 6)):
                at.append((b, rs.randint(h), rs.randint(rows), rs.randint(d)))
                kinds.append((math.nan, math.inf, -math.inf)[rs.randint(3)])
    places = torch.tensor(at, device="cuda").T
    where = (places[0], places[1], 1, places[2], places[3])
    tails[where] = 0.0
    clean = f.attend()
    f.check(clean, requests=range(0, r, 40))
    tails[where] = torch.tensor(kinds, device="cuda", dtype=torch.float32).to(dtype)
    values = tails[where].tolist()  # (of the same place twice: the one that is there)
    want = clean.clone()
    for (b, head, row, ch), v in zip(at, values):
        first = max(0, lens[b] // page * page + row - (lens[b] - new[b]))  # its first token that attends the position
        want[int(f.cu[b]) + first:int(f.cu[b + 1]), head * g:(head + 1) * g, ch] += v
    for _ in range(3):
        out = f.attend()
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf),
                           want.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf))
    assert not want.isfinite().all() and f.cache.status() == 0
    # and none of it is left behind for the next step
    tails[where] = 0.0
    assert torch.equal(f.attend(), clean) and f.cache.status() == 0
