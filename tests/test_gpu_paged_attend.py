"""Attention of several new tokens per request over the paged cache, against the
definition in 64 bits on the cache's own codes, scales and tails."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from bit_quantized_kv_kvq_gb300 import paged
from tests.test_gpu_paged import BF16, CODE, F16, ints
from tests.test_gpu_paged_state import Recorder, apart, capture

pytestmark = pytest.mark.gpu


class Filled:
    """A cache of one layer whose pages, scales and tails are random, for requests
    of the given lengths (after the step) with `new` tokens each."""

    def __init__(self, lens, new, hq, h, d, page, code, dtype, seed=0, pad=0, lead=0, slots=None):
        r = slots or len(lens)
        self.lens, self.new, self.hq, self.h, self.d, self.page, self.code, self.dtype = lens, new, hq, h, d, page, code, dtype
        rs = np.random.RandomState(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // page) for n in lens]
        mp, pages = max(need) + 1, sum(need) + 3
        self.cache = c = kvq.PagedKVCache(1, r, h, d, page, pages, mp, CODE[code], dtype)
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda")
        for p0 in range(0, pages, 4096):
            x = normal(min(4096, pages - p0), h, 2, page, d)
            codes = (x * 36).round().clamp(-127, 127).to(torch.int8) if code == "int8" else (
                (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            c.pages(0)[p0:p0 + len(x)] = codes
        c.scales(0).copy_((1 / 36 if code == "int8" else 1 / 120) * torch.exp(0.5 * normal(pages, h, 2)))
        c.tails(0).copy_(normal(r, h, 2, page, d))
        order, at = rs.permutation(pages), 0
        table = np.full((len(lens), mp), -1, np.int32)
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        self.table, self.dlens = ints(table), ints(lens)
        self.cu = np.concatenate([[0], np.cumsum(new)]) + lead
        self.dcu = ints(self.cu)
        self.tokens = int(self.cu[-1]) + pad
        self.q = normal(self.tokens, hq + 2 * h, d).to(dtype)[:, :hq]
        self.scale = 1 / math.sqrt(d)

    def attend(self, **kw):
        return self.cache.attend(0, kw.pop("q", self.q), self.dcu, self.table, self.dlens, kw.pop("scale", self.scale), **kw)

    def kv(self, b, head):
        """Keys and values of one head as attention reads them, fp64."""
        n, out = self.lens[b], []
        ids = self.table[b, :n // self.page].long()
        codes = self.cache.pages(0)
        codes = codes.view(torch.float8_e4m3fn) if self.code == "e4m3" else codes
        for i in range(2):
            x = codes[ids, head, i].float().double() * self.cache.scales(0)[ids, head, i].double()[:, None, None]
            out.append(torch.cat([x.reshape(-1, self.d), self.cache.tails(0)[b, head, i, :n % self.page].double()]))
        return out

    def check(self, out, q=None, scale=None, requests=None, weight=None):
        q, scale = (self.q if q is None else q).double(), self.scale if scale is None else scale
        u = torch.finfo(self.dtype).eps / 2
        g = self.hq // self.h
        for b in requests if requests is not None else range(len(self.lens)):
            n, m, lo = self.lens[b], self.new[b], int(self.cu[b])
            if m == 0:
                continue
            seen = torch.arange(n, device="cuda") <= n - m + torch.arange(m, device="cuda")[:, None]
            for head in range(self.h):
                k, v = self.kv(b, head)
                for a in range(head * g, (head + 1) * g):
                    x = q[lo:lo + m, a]
                    s = (x @ k.T * scale).masked_fill(~seen, -math.inf)
                    p = torch.softmax(s, 1)
                    ref, w = p @ v, p @ v.abs()
                    size = (x.abs() @ k.abs().T * scale).amax(1, keepdim=True)
                    # weights rounded to the input type (in fp16 those below its normal
                    # numbers to 2^-25, beside a sum of 2^6 or more), the
                    # scores' fp32 sums (256 roundings of 2^-23 of the sum of magnitudes), exponentials
                    # and sums, the output's own rounding
                    tol = ((weight or u) + 2 * 256 * 2.0 ** -23 * size + 2.0 ** -18) * w * 1.01 + u * ref.abs()
                    if self.dtype == F16:
                        tol += n * 2.0 ** -31 * v.abs().amax()
                    err = (out[lo:lo + m, a].double() - ref).abs()
                    assert (err <= tol).all(), (b, a, (err / tol).max().item())


CASES = [
    # lens, new, hq, h, d, page, code, dtype
    ([1], [1], 1, 1, 64, 16, "int8", F16),
    ([1, 2, 3], [1, 2, 1], 4, 2, 128, 16, "e4m3", BF16),
    ([16, 17, 15, 32], [16, 1, 3, 2], 8, 2, 128, 16, "int8", F16),
    ([100, 0, 257, 129, 128], [5, 0, 4, 129, 1], 8, 8, 128, 64, "int8", BF16),
    ([1000, 777, 1, 640, 513], [1, 6, 1, 3, 8], 32, 8, 128, 16, "int8", F16),
    ([1000, 777, 1, 640, 513], [1, 6, 1, 3, 8], 16, 4, 64, 32, "e4m3", BF16),
    ([2000, 1500, 300], [700, 1, 300], 12, 4, 128, 128, "e4m3", F16),
    ([2000, 1500, 300], [700, 0, 299], 10, 2, 64, 64, "int8", F16),
    ([1021], [509], 3, 3, 128, 32, "int8", F16),
    ([5000], [5], 6, 1, 128, 64, "e4m3", F16),
    ([5000, 4999], [33, 17], 16, 1, 64, 128, "int8", BF16),
    ([700, 30], [40, 30], 40, 2, 128, 16, "int8", F16),
    ([300, 130], [9, 130], 130, 1, 64, 16, "e4m3", F16),
    ([300, 200], [3, 1], 600, 2, 64, 64, "int8", BF16),
    ([9000], [9000], 2, 1, 64, 64, "int8", F16),
    ([40000, 3], [1, 2], 8, 1, 128, 128, "int8", F16),
    ([30000, 20000], [250, 9], 8, 2, 128, 64, "e4m3", BF16),
    (list(range(1, 80, 3)), [min(n, 1 + n % 5) for n in range(1, 80, 3)], 7, 7, 128, 16, "int8", F16),
    (list(range(130, 400, 7)), [n % 60 for n in range(130, 400, 7)], 14, 2, 64, 32, "e4m3", F16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%s-h%dx%d-d%d-p%d-%s" % (c[0][:3], c[1][:3], c[2], c[3], c[4], c[5], c[6]))
def test_attend(case):
    f = Filled(*case, seed=len(case[0]))
    launches = kvq.kernel_launches()
    out = f.attend()
    assert kvq.kernel_launches() == launches + 2
    f.check(out)
    assert torch.equal(out, f.attend())  # the same bits every time
    assert f.cache.status() == 0


@pytest.mark.parametrize("code,d", [("int8", 128), ("e4m3", 64)])
def test_weights_of_11_bits_in_bf16(code, d):
    """Tiles of complete pages take fp16 weights in a bf16 cache too."""
    f = Filled([2944, 640, 128], [100, 64, 1], 8, 2, d, 64, code, BF16, seed=12)
    f.check(f.attend(), weight=2.0 ** -11)
    # a scale beyond fp16 in one page: the bound of bf16 weights
    f.cache.scales(0)[f.table[0, 3].item(), :, 1] *= 2.0 ** 40
    f.check(f.attend())
    f.check(f.attend(), weight=2.0 ** -11, requests=[1, 2])


def test_single_tokens_agree_with_decode():
    """One token a request: both are within the bound of the definition."""
    lens = [1, 16, 17, 500, 0, 1024, 333]
    f = Filled(lens, [min(1, n) for n in lens], 8, 2, 128, 16, "int8", F16, seed=4)
    out = f.attend()
    f.check(out)
    live = torch.tensor([n > 0 for n in lens], device="cuda")
    q = torch.zeros(len(lens), 8, 128, dtype=F16, device="cuda")
    q[live] = f.q
    f.check(f.cache.decode(0, q, f.table, f.dlens, f.scale)[live])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_padded_batch(dtype):
    """Rows before, after and between requests' ranges are left as they are."""
    f = Filled([300, 70, 128], [60, 0, 9], 6, 2, 64, 32, "int8", dtype, pad=100, lead=37, slots=9)
    out = torch.full((f.tokens, 6, 64), 7.0, dtype=dtype, device="cuda")
    f.attend(out=out)
    f.check(out)
    assert (out[:37] == 7).all() and (out[37 + 69:] == 7).all()
    # a request whose range ends before it starts has none
    f.dcu = ints([97, 37, 97, 105])
    f.new, f.cu = [0, 60, 8], np.array([97, 37, 97, 105])
    out.fill_(7.0)
    f.attend(out=out)
    f.check(out)
    assert (out[:37] == 7).all() and (out[105:] == 7).all() and f.cache.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", [0, 1])
def test_later_tokens_of_the_open_page_do_not_reach_earlier_ones(d, value, which):
    f = Filled([290, 100], [60, 40], 4, 2, d, 64, "int8", F16, seed=2)
    want = f.attend()
    row = 279 - 256  # position 279 of request 0, channel 5 of head 1
    f.cache.tails(0)[0, 1, which, row, 5] = value
    out = f.attend()
    first = 279 - 230  # the token at that position
    assert torch.equal(out[:first], want[:first]) and torch.equal(out[60:], want[60:])
    assert torch.equal(out[:, :2], want[:, :2])
    bad = ~out[first:60, 2:].isfinite()
    assert (bad[..., 5].all() and bad.sum() == bad[..., 5].sum()) if which else bad.any(-1).sum() > 0
    if which and not math.isnan(value):
        assert (out[first:60, 2:, 5] == value).all()
    assert f.cache.status() == 0


@pytest.mark.parametrize("d,dtype,code", [(128, F16, "int8"), (64, BF16, "e4m3"), (128, BF16, "int8"), (64, F16, "e4m3")])
def test_scales_of_any_kind(d, dtype, code):
    """Zero, tiny and huge scales; a page that reads as NaN reaches the rows that attend any of it."""
    f = Filled([400], [120], 4, 2, d, 16, code, dtype, seed=3)
    c, ids = f.cache, f.table[0].tolist()
    c.scales(0)[ids[3]] = 0.0
    c.pages(0)[ids[3]] = 0
    c.scales(0)[ids[5], :, 1] *= 2.0 ** -16
    c.scales(0)[ids[6], :, 0] *= 2.0 ** -20
    c.scales(0)[ids[7], :, 1] *= 2.0 ** 9
    f.check(f.attend())
    if dtype == BF16:
        c.scales(0)[ids[8], :, 1] *= 2.0 ** -100
        c.scales(0)[ids[9], :, 1] *= 2.0 ** 80
        f.check(f.attend())
    want = f.attend()
    for i in range(2):
        for bad in (math.nan, math.inf):
            kept = c.scales(0)[ids[19], 1, i].item()
            c.scales(0)[ids[19], 1, i] = bad
            if bad == math.inf:
                kept_codes = c.pages(0)[ids[19], 1, i].clone()
                c.pages(0)[ids[19], 1, i] = 0
                if code == "e4m3":
                    c.pages(0)[ids[19], 1, i, 4, 9] = 127
            out = f.attend()
            c.scales(0)[ids[19], 1, i] = kept
            if bad == math.inf:
                c.pages(0)[ids[19], 1, i] = kept_codes
            first = 19 * 16 - 280  # the first token that attends the page
            assert torch.equal(out[:first], want[:first]) and torch.equal(out[:, :2], want[:, :2])
            assert out[first:, 2:].isnan().all()
    assert c.status() == 0


@pytest.mark.parametrize("lens,new", [([500], [37]), ([500], [400])])
def test_a_scale_of_zero_gives_the_mean(lens, new):
    f = Filled(lens, new, 4, 1, 64, 64, "e4m3", F16)
    f.check(f.attend(scale=0.0), scale=0.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,top", [(F16, 61440.0), (BF16, 2.0 ** 55)])
def test_scores_of_any_size(dtype, top, d):
    """Scores far past where a last place of theirs is worth a weight: rows are finite
    means of values, and the largest score's where it stands out."""
    n, m = 333, 40
    f = Filled([n], [m], 2, 1, d, 64, "int8", dtype, seed=5)
    q = torch.full((m, 2, d), top, dtype=dtype, device="cuda")
    f.cache.pages(0)[:, :, 0] = 0
    f.cache.pages(0)[f.table[0, 2].item(), :, 0, 9] = 100  # position 137
    f.cache.scales(0)[:, :, 0] = 1.0
    f.cache.tails(0)[:, :, 0] = 0
    v = f.kv(0, 0)[1]
    for sign in (1, -1):
        out = f.attend(q=sign * q, scale=0.5).double()
        for i in range(0, m, 7):
            ref = v[137] if sign > 0 else torch.cat([v[:137], v[138:n - m + i + 1]]).mean(0)
            tol = 2 * torch.finfo(dtype).eps * v.abs().mean(0).clamp(min=ref.abs())
            assert ((out[i] - ref).abs() <= tol).all(), (sign, i)


@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_beside_a_large_one(d):
    """A first token of e^13 times the weight of each other one, which hold the values."""
    n = 3000
    f = Filled([n], [10], 2, 1, d, 64, "int8", F16, seed=6)
    c = f.cache
    c.pages(0).zero_()
    c.scales(0).fill_(1.0)
    c.tails(0).zero_()
    c.pages(0)[f.table[0, 0].item(), 0, 0, 0, 0] = 13
    c.pages(0)[:, 0, 1] = 1
    c.tails(0)[:, :, 1] = 1
    c.pages(0)[f.table[0, 0].item(), 0, 1, 0] = 0
    q = torch.zeros(10, 2, d, dtype=F16, device="cuda")
    q[..., 0] = 1
    out = f.attend(q=q, scale=1.0).double()
    for i in range(10):
        small = (n - 10 + i) * math.exp(-13.0)
        ref = small / (1 + small)
        assert ((out[i] - ref).abs() <= (2.0 ** -10 + 2.0 ** -14) * ref).all()


def test_what_the_device_finds_bad():
    """Lengths, ranges and pages out of bounds are left out; the other requests have their rows."""
    def fresh():
        return Filled([300, 200, 150], [50, 20, 30], 4, 2, 64, 32, "int8", F16, seed=9)
    want = fresh().attend()
    for what in ("length", "negative length", "short length", "range", "negative range"):
        f = fresh()
        cu, lens = f.cu.tolist(), list(f.lens)
        others = [0, 2]
        if what == "length":
            lens[1] = f.table.shape[1] * 32 + 1
        elif what == "negative length":
            lens[1] = -5
        elif what == "short length":
            lens[1] = 19
        elif what == "range":
            cu[3], others = 101, [0, 1]
        else:
            cu[0], others = -1, [1, 2]
        f.dcu, f.dlens = ints(cu), ints(lens)
        out = torch.full_like(want, 7.0)
        f.attend(out=out)
        for b in range(3):
            rows = slice(int(f.cu[b]), int(f.cu[b + 1]))
            assert torch.equal(out[rows], want[rows]) if b in others else (out[rows] == 7).all(), (what, b)
        with pytest.raises(kvq.KVQError) as e:
            f.cache.status()
        assert e.value.status == 7
    for bad in (-1, 1 << 30):
        f = fresh()
        f.table[1, 2] = bad
        out = f.attend()
        for b in (0, 2):
            assert torch.equal(out[int(f.cu[b]):int(f.cu[b + 1])], want[int(f.cu[b]):int(f.cu[b + 1])])
        with pytest.raises(kvq.KVQError):
            f.cache.status()
    # entries of pages past the length are not read
    f = fresh()
    f.table[:, -1] = 1 << 30
    assert torch.equal(f.attend(), want) and f.cache.status() == 0


def test_streams_and_graphs_have_workspaces_of_their_own(monkeypatch):
    f = Filled([20000, 33, 600], [20, 33, 1], 8, 2, 128, 32, "int8", F16, seed=8)
    qs = [torch.randn(54, 8, 128, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(4)]
    want = [f.attend(q=q) for q in qs]
    rec = Recorder(paged._lib)
    seen = []
    def call(*args):
        seen.append((args[12], args[12] + args[13]))
        return rec.lib.kvq_paged_attention(*args)
    class Lib:
        def __getattr__(self, name):
            return call if name == "kvq_paged_attention" else getattr(rec.lib, name)
    monkeypatch.setattr(paged, "_lib", Lib())
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want[0]) for _ in qs]
    torch.cuda.synchronize()
    for i, st in ((0, side), (1, other)):
        f.attend(q=qs[i], out=outs[i], stream=st)
    graphs = [capture(side, lambda i=i: f.attend(q=qs[i], out=outs[i], stream=side)) for i in (2, 3)]
    assert len(seen) == 4 and apart(seen)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for i, st in ((0, side), (1, other)):
            f.attend(q=qs[i], out=outs[i], stream=st)
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert f.cache.status() == 0


def test_lengths_that_change_under_a_captured_call():
    """One graph serves steps of other lengths and token counts."""
    f = Filled([5000, 3000, 64], [40, 1, 23], 8, 2, 128, 64, "e4m3", BF16, seed=1)
    out = torch.zeros(f.tokens, 8, 128, dtype=BF16, device="cuda")
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        f.attend(out=out)
    for lens, new in (([5000, 3000, 64], [40, 1, 23]), ([700, 1, 0], [60, 1, 0]), ([12, 2900, 64], [1, 2, 61]), ([0, 0, 0], [0, 0, 0])):
        f.lens, f.new, f.cu = lens, new, np.concatenate([[0], np.cumsum(new)])
        f.dlens.copy_(ints(lens))
        f.dcu.copy_(ints(f.cu))
        out.fill_(3.0)
        gr.replay()
        f.check(out)
        assert (out[sum(new):] == 3).all()
    assert f.cache.status() == 0


def test_pages_past_four_gibibytes():
    h, d, page = 8, 128, 128
    pages = (1 << 32) // (h * 2 * page * d) + 40
    cache = kvq.PagedKVCache(1, 1, h, d, page, pages, 4)
    small = kvq.PagedKVCache(1, 1, h, d, page, 4, 4)
    k, v = (torch.randn(300, h, d, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2))
    q = torch.randn(120, h, d, generator=torch.Generator().manual_seed(3)).half().cuda()
    outs = []
    for c, ids in ((cache, [5, pages - 1, pages - 2]), (small, [2, 1, 0])):
        n = c.cfg.num_pages
        table, free = ints([[-1] * 4]), ints(np.zeros(n))
        free[:3] = ints(ids)
        plan = c.reserve(ints([0]), ints([300]), table, free, ints([3]), 300)
        c.write(0, k, v, plan.cu_tokens, plan.slots, plan.lens)
        outs.append(c.attend(0, q, ints([0, 120]), table, plan.lens, 0.1))
        assert c.status() == 0
    assert torch.equal(*outs) and outs[0].any()


def test_many_requests():
    """4096 slots, most of them idle or short."""
    rs = np.random.RandomState(5)
    lens = rs.randint(0, 30, 4096)
    new = np.minimum(lens, rs.randint(0, 4, 4096))
    lens[[3, 4095]], new[[3, 4095]] = [700, 90], [300, 1]
    f = Filled(lens.tolist(), new.tolist(), 4, 2, 64, 16, "int8", F16, seed=1)
    out = f.attend()
    f.check(out, requests=list(np.flatnonzero(new)[:25]) + [3, 4095])
    assert f.cache.status() == 0


@pytest.mark.parametrize("sizes", [[200, 1, 1, 130, 17], [349], [64, 64, 64, 157]])
def test_a_prompt_in_chunks(sizes):
    """Served a chunk at a time: planned, normalised and rotated, written, attended;
    every chunk's rows are the definition's on the cache as it stands then."""
    r, hq, h, d, page = 3, 8, 2, 128, 32
    gen = torch.Generator().manual_seed(sum(sizes) + len(sizes))
    cache = kvq.PagedKVCache(1, r, h, d, page, 60, 20, kvq.PAGE_INT8, F16)
    table, free, count, lens = ints(np.full((r, 20), -1)), ints(np.arange(60)), ints([60]), ints([0] * r)
    rot, w = kvq.Rotation.standard(d), torch.rand(2, d, generator=gen).add(0.5).cuda()
    shared = ints([0] * 60)
    f = Filled.__new__(Filled)
    f.__dict__.update(cache=cache, hq=hq, h=h, d=d, page=page, code="int8", dtype=F16, table=table, scale=0.09)
    have = [0] * r
    for step, size in enumerate(sizes):
        new = [size, step % 2, 0 if step else 50]
        t = sum(new)
        x = torch.randn(t, hq + 2 * h, d, generator=gen).half().cuda()
        plan = cache.reserve(lens, ints(new), table, free, count, t, lens_out=lens, free_count_out=count)
        q, k = kvq.norm_rotate(x[:, :hq], x[:, hq:hq + h], plan.positions, rot, w[0], w[1])
        cache.write(0, k, x[:, hq + h:], plan.cu_tokens, plan.slots, plan.lens)
        out = cache.attend(0, q, plan.cu_tokens, table, plan.lens, 0.09)
        have = [a + b for a, b in zip(have, new)]
        f.__dict__.update(lens=have, new=new, cu=np.concatenate([[0], np.cumsum(new)]), q=q)
        f.check(out)
    # slot 2 ends, becomes a branch of slot 0; both go on by the same tokens and get the same bits
    cache.release(ints([0, 0, 1]), lens, table, free, count, shared=shared)
    cache.fork(ints([0]), ints([2]), lens, table, free, count, shared)
    assert lens.tolist() == [have[0], have[1], have[0]]
    for m in (3, 40):
        x = torch.randn(m, hq + 2 * h, d, generator=gen).half().cuda()
        x = torch.cat([x, x])
        plan = cache.reserve(lens, ints([m, 0, m]), table, free, count, 2 * m, lens_out=lens, free_count_out=count)
        q, k = kvq.norm_rotate(x[:, :hq], x[:, hq:hq + h], plan.positions, rot, w[0], w[1])
        cache.write(0, k, x[:, hq + h:], plan.cu_tokens, plan.slots, plan.lens)
        out = cache.attend(0, q, plan.cu_tokens, table, plan.lens, 0.09)
        have = [have[0] + m, have[1], have[0] + m]
        f.__dict__.update(lens=have, new=[m, 0, m], cu=np.array([0, m, m, 2 * m]), q=q)
        f.check(out)
    cache.release(ints([1, 1, 0]), lens, table, free, count, shared=shared)
    cache.release(ints([0, 0, 1]), lens, table, free, count, shared=shared)
    assert count.item() == 60 and not shared.any() and not lens.any() and cache.status() == 0
    assert sorted(free.tolist()) == list(range(60))


def test_refusals():
    f = Filled([50], [20], 4, 2, 64, 16, "int8", F16)
    c, q = f.cache, f.q.contiguous()
    ws = torch.empty(c.workspace_bytes(4, attend=True), dtype=torch.uint8, device="cuda")
    go = lambda q=q, cu=f.dcu, table=f.table, lens=f.dlens, scale=0.1, layer=0, **kw: c.attend(layer, q, cu, table, lens, scale, **kw)
    for bad in (lambda: go(q=q.float()), lambda: go(q=q.bfloat16()), lambda: go(q=q.cpu()), lambda: go(cu=f.dcu.long()),
                lambda: go(lens=f.dlens.float()), lambda: go(workspace=ws.cpu())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: go(q=q[..., :32]), lambda: go(cu=ints([0])), lambda: go(table=f.table[:, 1:].contiguous()),
                lambda: go(out=torch.zeros(20, 4, 64, device="cuda")), lambda: go(out=torch.zeros(19, 4, 64, dtype=F16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: go(q=q[:, :3].contiguous()), lambda: go(scale=-0.1), lambda: go(scale=math.nan), lambda: go(scale=math.inf),
                lambda: go(layer=1), lambda: go(layer=-1), lambda: go(workspace=ws[:-16])):
        with pytest.raises(kvq.KVQError):
            bad()
    assert go(q=q[:0]).shape == (0, 4, 64)
    f.check(go(workspace=ws, scale=f.scale))
    assert c.status() == 0
