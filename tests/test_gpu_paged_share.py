"""Forks of paged requests and the release of pages with several holders: the
books and the tails equal to the oracle's, refusals that change nothing."""
import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from oracle import paged_oracle as PO
from tests.test_gpu_paged import BF16, F16, ints

pytestmark = pytest.mark.gpu


class Books:
    """A table of requests without shared pages, some of them empty."""

    def __init__(self, r, page, longest, empty, seed, spare=9):
        rs = self.rs = np.random.RandomState(seed)
        self.page = page
        self.lens = rs.randint(1, longest + 1, r)
        self.lens[rs.permutation(r)[:empty]] = 0
        need = -(-self.lens // page)
        mp = longest // page + 2
        pages = int(need.sum()) + empty + spare
        order, at = rs.permutation(pages), 0
        self.table = np.full((r, mp), -3, np.int32)
        for b in range(r):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.free = np.full(pages, -5, np.int32)
        self.free[:pages - at] = order[at:]
        self.count = pages - at
        self.shared = np.zeros(pages, np.int32)

    def cache(self, layers=1, heads=1, dim=64, dtype=F16):
        self.c = kvq.PagedKVCache(layers, len(self.lens), heads, dim, self.page, len(self.free), self.table.shape[1],
                                  dtype=dtype)
        for i in range(layers):
            t = self.c.tails(i)
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).to(dtype))
        self.put()
        return self.c

    def put(self):
        self.d = dict(lens=ints(self.lens), table=ints(self.table), free=ints(self.free), count=ints([self.count]),
                      shared=ints(self.shared))

    def check(self):
        for k, want in (("lens", self.lens), ("table", self.table), ("free", self.free), ("count", [self.count]),
                        ("shared", self.shared)):
            assert np.array_equal(self.d[k].cpu().numpy(), np.asarray(want)), k

    def call_fork(self, src, dst):
        d = self.d
        self.c.fork(ints(src), ints(dst), d["lens"], d["table"], d["free"], d["count"], d["shared"])

    def fork(self, src, dst):
        src, dst = np.asarray(src), np.asarray(dst)
        self.call_fork(src, dst)
        self.lens, self.table, self.count, self.shared = PO.fork(src, dst, self.lens, self.table, self.free, self.count,
                                                                 self.shared, self.page)

    def release(self, done):
        d = self.d
        self.c.release(ints(done), d["lens"], d["table"], d["free"], d["count"], shared=d["shared"])
        self.lens, self.free, self.count, self.shared = PO.release_shared(np.asarray(done), self.lens, self.table, self.free,
                                                                          self.count, self.shared, self.page)


FORKS = [(2, 16, 5, 1, 1, 1, 64, F16), (9, 16, 200, 4, 2, 2, 64, BF16), (40, 64, 1000, 30, 3, 8, 128, F16),
         (7, 128, 127, 3, 5, 1, 128, BF16), (300, 32, 500, 250, 1, 1, 64, F16), (4096, 16, 40, 3000, 1, 1, 64, F16),
         (3, 16, 20000, 2, 1, 1, 64, F16)]


@pytest.mark.parametrize("r,page,longest,empty,layers,heads,dim,dtype", FORKS)
def test_fork(r, page, longest, empty, layers, heads, dim, dtype):
    bk = Books(r, page, longest, empty, r + page)
    c = bk.cache(layers, heads, dim, dtype)
    dst = bk.rs.permutation(np.flatnonzero(bk.lens == 0))
    src = bk.rs.choice(np.flatnonzero(bk.lens > 0), len(dst))
    src[::5] = -1  # pairs that are left out
    if len(src) > 2:
        src[1] = src[2]
    before = [c.tails(i).clone() for i in range(layers)]
    pages = [c.pages(i).clone() for i in range(layers)]
    launches = kvq.kernel_launches()
    n = bk.lens.copy()
    bk.fork(src, dst)
    tails = len(src) * layers * heads * 2 * page * dim * 2
    assert kvq.kernel_launches() == launches + (1 if tails <= 131072 else 2)
    bk.check()
    for i in range(layers):
        want = before[i]
        for s, t in zip(src, dst):
            if s >= 0:
                want[t, :, :, :n[s] % page] = want[s, :, :, :n[s] % page]
        assert torch.equal(c.tails(i), want) and torch.equal(c.pages(i), pages[i])
    assert c.status() == 0


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("why", ["source", "destination", "negative destination", "itself", "not empty", "twice", "length",
                                 "negative length", "pages", "count", "popped page"])
def test_a_refused_fork_changes_nothing(why, many):
    """One launch and two."""
    bk = Books(60 if many else 6, 16, 100, 40 if many else 3, 3)
    e, f = np.flatnonzero(bk.lens == 0), np.flatnonzero(bk.lens > 0)
    bk.lens[f] += bk.lens[f] % 16 == 0  # all have open pages
    src, dst = np.array([f[0], f[1], f[0]]), e[:3].copy()
    status = 7
    if why == "source":
        src[1] = len(bk.lens)
    elif why == "destination":
        dst[1] = len(bk.lens)
    elif why == "negative destination":
        dst[2] = -1
    elif why == "itself":
        dst[1] = src[1] = e[1]
    elif why == "not empty":
        dst[0] = f[2]
    elif why == "twice":
        dst[2] = dst[0]
    elif why == "length":
        bk.lens[f[1]] = bk.table.shape[1] * 16 + 1
    elif why == "negative length":
        bk.lens[f[1]] = -1
    elif why == "pages":
        bk.count, status = 2, 4
    elif why == "count":
        bk.count = len(bk.free) + 1
    else:
        bk.free[bk.count - 2] = len(bk.free)
    c = bk.cache(4 if many else 1, 4 if many else 1, 128 if many else 64)
    before = c.buffer.clone()
    bk.call_fork(src, dst)
    bk.check()
    with pytest.raises(kvq.KVQError) as err:
        c.status()
    assert err.value.status == status
    assert torch.equal(c.buffer, before)


def test_fork_copies_an_entry_out_of_range_and_says_so():
    bk = Books(4, 16, 100, 1, 8)
    s, e = int(np.argmax(bk.lens)), int(np.argmin(bk.lens))
    bk.table[s, 1] = 1 << 20
    c = bk.cache()
    bk.call_fork([s], [e])
    n = int(bk.lens[s])
    assert bk.d["lens"][e].item() == n and bk.d["table"][e, 1].item() == 1 << 20
    want = bk.shared.copy()
    want[bk.table[s, :n // 16][bk.table[s, :n // 16] != 1 << 20]] += 1
    assert np.array_equal(bk.d["shared"].cpu().numpy(), want)
    with pytest.raises(kvq.KVQError):
        c.status()


@pytest.mark.parametrize("r,page,longest", [(4, 16, 50), (30, 64, 3000), (500, 16, 400), (4096, 16, 60), (12, 16, 60000)])
@pytest.mark.parametrize("ending", [0.3, 1.0])
def test_release_of_shared_pages(r, page, longest, ending):
    """Branches of branches, released a part at a time until none is left."""
    bk = Books(r, page, longest, r // 2, r)
    c = bk.cache()
    pages = len(bk.free)
    for _ in range(2):
        e, f = np.flatnonzero(bk.lens == 0), np.flatnonzero(bk.lens > 0)
        dst = bk.rs.permutation(e)[:(len(e) + 1) // 2]
        bk.fork(bk.rs.choice(f, len(dst)), dst)
        bk.check()
    while bk.lens.any():
        live = np.flatnonzero(bk.lens)
        done = np.zeros(r, np.int64)
        done[bk.rs.permutation(live)[:max(1, int(ending * len(live)))]] = 1
        if len(live) < 4:
            done[:] = 1
        launches = kvq.kernel_launches()
        bk.release(done)
        assert kvq.kernel_launches() == launches + 1
        bk.check()
    assert bk.count == pages and not bk.shared.any() and c.status() == 0
    assert sorted(bk.free.tolist()) == list(range(pages))


def test_release_without_sharing_is_the_plain_release():
    bk = Books(50, 32, 900, 10, 4)
    c = bk.cache()
    done = bk.rs.randint(0, 2, 50)
    plain = {k: v.clone() for k, v in bk.d.items()}
    c.release(ints(done), plain["lens"], plain["table"], plain["free"], plain["count"])
    bk.release(done)
    bk.check()
    for k in ("lens", "free", "count"):
        assert torch.equal(plain[k], bk.d[k])
    assert c.status() == 0


def test_release_of_bad_books():
    # a page released more often than held goes back once
    c = kvq.PagedKVCache(1, 3, 1, 64, 16, 6, 4)
    table, free, count, shared = ints([[0, 1, -1, -1], [1, 2, -1, -1], [1, 9, -1, -1]]), ints([5, -1, -1, -1, -1, -1]), ints([1]), ints([0] * 6)
    lens = ints([32, 20, 30])
    c.release(ints([1, 1, 0]), lens, table, free, count, shared=shared)
    assert count.item() == 4 and free.tolist()[:4] == [5, 0, 1, 2] and not shared.any() and lens.tolist() == [0, 0, 30]
    with pytest.raises(kvq.KVQError) as e:
        c.status()
    assert e.value.status == 7
    # an entry out of range is left out
    c.release(ints([0, 0, 1]), lens, table, free, ints([1]), shared=shared)
    assert free.tolist()[:2] == [5, 1] and not lens.any()
    with pytest.raises(kvq.KVQError):
        c.status()
    # pages past the stack's room are dropped; a count out of range changes nothing
    lens, count = ints([32, 0, 0]), ints([5])
    c.release(ints([1, 0, 0]), lens, table, free, count, shared=shared)
    assert count.item() == 6 and free[5].item() == 0
    with pytest.raises(kvq.KVQError):
        c.status()
    lens, count, kept = ints([32, 0, 0]), ints([7]), free.clone()
    c.release(ints([1, 0, 0]), lens, table, free, count, shared=shared)
    assert lens.tolist() == [32, 0, 0] and count.item() == 7 and torch.equal(free, kept)
    with pytest.raises(kvq.KVQError):
        c.status()
    # a length out of range: the other requests end
    lens, count = ints([-1, 20, 65]), ints([0])
    c.release(ints([1, 1, 1]), lens, table, free, count, shared=ints([0] * 6))
    assert not lens.any() and count.item() == 2 and free.tolist()[:2] == [1, 2]
    with pytest.raises(kvq.KVQError):
        c.status()


@pytest.mark.parametrize("r,longest", [(6, 90), (300, 400)])
def test_fork_and_release_from_a_graph(r, longest):
    """A captured branch and end, replayed on the books as they are; a release by one CTA and by a cluster."""
    bk = Books(r, 16, longest, 3, 2)
    c = bk.cache(2, 2)
    e, f = np.flatnonzero(bk.lens == 0), np.flatnonzero(bk.lens > 0)
    src, dst, done = ints([f[0], f[1], -1]), ints(e), ints((np.arange(r) == e[0]) | (np.arange(r) % 2 == f[0] % 2))
    keep = {k: v.clone() for k, v in bk.d.items()}
    d = bk.d
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        c.fork(src, dst, d["lens"], d["table"], d["free"], d["count"], d["shared"])
        c.release(done, d["lens"], d["table"], d["free"], d["count"], shared=d["shared"])
    first = [bk.lens, bk.table, bk.free, bk.count, bk.shared]
    for _ in range(3):
        for k, v in keep.items():
            d[k].copy_(v)
        bk.lens, bk.table, bk.free, bk.count, bk.shared = first
        gr.replay()
        args = (np.array([f[0], f[1], -1]), e)
        bk.lens, bk.table, bk.count, bk.shared = PO.fork(*args, bk.lens, bk.table, bk.free, bk.count, bk.shared, 16)
        bk.lens, bk.free, bk.count, bk.shared = PO.release_shared(done.cpu().numpy(), bk.lens, bk.table, bk.free, bk.count,
                                                                  bk.shared, 16)
        bk.check()
    assert c.status() == 0


def test_refusals_of_the_binding():
    bk = Books(4, 16, 50, 1, 1)
    c, d = bk.cache(), bk.d
    ok = ints([0])
    for bad in (dict(src=ok.long()), dict(src=ok.cpu()), dict(shared=d["shared"].float())):
        with pytest.raises(TypeError):
            a = {**dict(src=ok, dst=ok, shared=d["shared"]), **bad}
            c.fork(a["src"], a["dst"], d["lens"], d["table"], d["free"], d["count"], a["shared"])
    for bad in (dict(dst=ints([0, 1])), dict(shared=d["shared"][1:]), dict(src=ints([[0]]))):
        with pytest.raises(ValueError):
            a = {**dict(src=ok, dst=ok, shared=d["shared"]), **bad}
            c.fork(a["src"], a["dst"], d["lens"], d["table"], d["free"], d["count"], a["shared"])
    with pytest.raises(ValueError):
        c.release(ints([0] * 4), d["lens"], d["table"], d["free"], d["count"], shared=d["shared"][1:])
    with pytest.raises(kvq.KVQError):
        c.fork(ints([0] * 5), ints([1] * 5), d["lens"], d["table"], d["free"], d["count"], d["shared"])  # more pairs than slots
    c.fork(ok[:0], ok[:0], d["lens"], d["table"], d["free"], d["count"], d["shared"])  # nothing to do
    bk.check()
    assert c.status() == 0
