"""Drafted tokens that are taken back: inside the open page by the length alone, to its start with its
page, and past it by a fork. The request goes on as one that never had them, to the bit."""
import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from tests.test_gpu_paged import BF16, F16, ints

pytestmark = pytest.mark.gpu

PAGE, PAGES, ROW = 32, 40, 12


class Serve:
    """One layer; tokens of a request by their position and a variant, so that two caches get the same."""

    def __init__(self, d, code, dtype):
        self.d, self.dtype = d, dtype
        self.cache = kvq.PagedKVCache(1, 2, 2, d, PAGE, PAGES, ROW, code, dtype)
        self.lens, self.table = ints([0, 0]), ints(np.full((2, ROW), -1))
        self.free, self.count, self.shared = ints(np.arange(PAGES)), ints([PAGES]), ints([0] * PAGES)

    def step(self, slot, n, variant=0):
        have = self.lens[slot].item()
        gen = torch.Generator().manual_seed(variant)
        x = torch.randn(400, 8, self.d, generator=gen)[have:have + n].to(self.dtype).cuda()
        new = ints([n if b == slot else 0 for b in range(2)])
        plan = self.cache.reserve(self.lens, new, self.table, self.free, self.count, n, lens_out=self.lens,
                                  free_count_out=self.count)
        self.cache.write(0, x[:, 4:6], x[:, 6:], plan.cu_tokens, plan.slots, plan.lens)
        return self.cache.attend(0, x[:, :4], plan.cu_tokens, self.table, self.lens, 0.1)

    def end(self):
        self.cache.release(ints([1, 1]), self.lens, self.table, self.free, self.count, shared=self.shared)
        assert self.count.item() == PAGES and sorted(self.free.tolist()) == list(range(PAGES))
        assert self.cache.status() == 0


KINDS = [(64, kvq.PAGE_INT8, F16), (128, kvq.PAGE_E4M3, BF16)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "d%d" % k[0])
@pytest.mark.parametrize("have,drafts,kept", [(37, 8, 3), (37, 8, 0), (33, 20, 1), (30, 12, 5), (64, 9, 2), (1, 30, 0)])
def test_inside_the_open_page(kind, have, drafts, kept):
    """Drafts may have completed a page, if those taken back are all behind it."""
    a, b = Serve(*kind), Serve(*kind)
    for s in (a, b):
        s.step(0, have)
    a.step(0, drafts)
    assert have + kept > (have + drafts) // PAGE * PAGE
    a.lens[0] = have + kept
    if kept:
        b.step(0, kept)
    for n in (1, 40, 3):
        assert torch.equal(a.step(0, n, 1), b.step(0, n, 1))
    assert torch.equal(a.count, b.count) and torch.equal(a.lens, b.lens)
    a.end(), b.end()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "d%d" % k[0])
@pytest.mark.parametrize("have,drafts", [(64, 7), (60, 12), (61, 4)])
def test_to_the_start_of_the_open_page(kind, have, drafts):
    a, b = Serve(*kind), Serve(*kind)
    for s in (a, b):
        s.step(0, have)
    a.step(0, drafts)
    k = (have + drafts) // PAGE
    a.lens[0] = k * PAGE
    a.free[a.count.item()] = a.table[0, k]
    a.count += 1
    if k * PAGE > have:
        b.step(0, k * PAGE - have)
    for n in (1, 40):
        assert torch.equal(a.step(0, n, 1), b.step(0, n, 1))
    assert torch.equal(a.count, b.count)
    a.end(), b.end()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "d%d" % k[0])
@pytest.mark.parametrize("accepted", [True, False])
def test_drafts_in_a_fork(kind, accepted):
    a, b = Serve(*kind), Serve(*kind)
    for s in (a, b):
        s.step(0, 90)
    a.cache.fork(ints([0]), ints([1]), a.lens, a.table, a.free, a.count, a.shared)
    drafted = a.step(1, 50)
    slot = 1 if accepted else 0
    a.cache.release(ints([accepted, not accepted]), a.lens, a.table, a.free, a.count, shared=a.shared)
    if accepted:
        assert torch.equal(drafted, b.step(0, 50))
    for n in (1, 40):
        assert torch.equal(a.step(slot, n, 1), b.step(0, n, 1))
    assert not a.shared.any() and torch.equal(a.count, b.count)
    a.end(), b.end()
