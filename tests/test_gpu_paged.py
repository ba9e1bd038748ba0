"""The paged 8-bit cache on the GPU against its oracle: plans and codes equal,
decode attention within a bound derived from its roundings; ranges that the
device finds bad; serving steps, captured and replayed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

CODE = {"int8": kvq.PAGE_INT8, "e4m3": kvq.PAGE_E4M3}
F16, BF16 = torch.float16, torch.bfloat16


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def decode_bound(w, size, vmax, n, out_eps, ref):
    """|o - ref| allowed: weights rounded to fp16 (2^-11 each, or 2^-25 of the
    largest below fp16's normal range, of at least 2^-8 of the sum's unit), the
    fp32 score sums (at most 256 roundings of 2^-23 each, on the sum of
    magnitudes), and the output's own rounding."""
    return (2.0 ** -11 + 2 * 256 * 2.0 ** -23 * size + 2.0 ** -18) * w * 1.01 + n * 2.0 ** -25 * vmax + out_eps * np.abs(ref)


# -- planning ----------------------------------------------------------------
PLANS = [(1, 16, 1, 5), (7, 64, 40, 300), (33, 32, 3000, 200), (512, 16, 5000, 100), (1500, 128, 20000, 90),
         (4096, 16, 4096, 40)]


@pytest.mark.parametrize("r,page,tokens,longest", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve_and_release(r, page, tokens, longest, in_place):
    rs = np.random.RandomState(r + page)
    lens = rs.randint(0, longest, r)
    lens[rs.randint(r)] = 0
    new = rs.multinomial(tokens - tokens // 3, np.ones(r) / r)
    new[rs.permutation(r)[:r // 3]] = 0
    mp = int((lens + new).max()) // page + 2
    used = -(-lens // page)
    pages = int((-(-(lens + new) // page)).sum()) + 3
    order = rs.permutation(pages)
    table = np.full((r, mp), -7, np.int32)
    at = 0
    for b in range(r):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    free = np.zeros(pages, np.int32)
    free[:pages - at] = order[at:]
    cache = kvq.PagedKVCache(1, r, 1, 64, page, pages, mp)
    dl, dt, df, dc = ints(lens), ints(table), ints(free), ints([pages - at])
    kw = dict(lens_out=dl, free_count_out=dc) if in_place else {}
    launches = kvq.kernel_launches()
    plan = cache.reserve(dl, ints(new), dt, df, dc, tokens, **kw)
    assert kvq.kernel_launches() == launches + (1 if tokens <= 4096 else 2)
    want = PO.reserve(lens, new, table, free, pages - at, tokens, page)
    for got, ref in zip((dt, plan.cu_tokens, plan.slots, plan.positions, plan.lens, plan.free_count), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref)), ref)
    if not in_place:
        assert np.array_equal(dl.cpu().numpy(), lens) and dc.item() == pages - at
    done = rs.randint(0, 2, r)
    lens2, free2, count2 = plan.lens.clone(), df.clone(), plan.free_count.clone()
    cache.release(ints(done), lens2, dt, free2, count2)
    wl, wf, wc = PO.release(done, want[4], want[0], free, want[5], page)
    assert np.array_equal(lens2.cpu().numpy(), wl) and count2.item() == wc
    assert np.array_equal(free2.cpu().numpy()[:wc], wf[:wc])
    assert cache.status() == 0


@pytest.mark.parametrize("why", ["pages", "row", "tokens", "negative add", "negative length", "count", "huge add"])
def test_reserve_that_does_not_fit_changes_nothing(why):
    cache = kvq.PagedKVCache(1, 3, 1, 64, 16, 20, 4)
    lens, new, count, tokens = [10, 0, 32], [1, 30, 2], [5], 40
    if why == "pages":
        count = [2]
    elif why == "row":
        new[2] = 33
    elif why == "tokens":
        tokens = 32
    elif why == "negative add":
        new[0] = -1
    elif why == "negative length":
        lens[1] = -3
    elif why == "count":
        count = [21]
    else:
        new[1] = 2 ** 31 - 1
    table = np.arange(12).reshape(3, 4)
    dt, df = ints(table), ints(np.arange(20))
    plan = cache.reserve(ints(lens), ints(new), dt, df, ints(count), tokens)
    torch.cuda.synchronize()
    assert np.array_equal(dt.cpu().numpy(), table)
    assert plan.cu_tokens.tolist() == [0] * 4 and plan.lens.tolist() == lens and plan.free_count.tolist() == count
    assert plan.slots.tolist() == [-1] * tokens and plan.positions.tolist() == [-1] * tokens
    with pytest.raises(kvq.KVQError) as e:
        cache.status()
    assert e.value.status == (4 if why in ("pages", "row", "tokens", "huge add") else 7)
    assert cache.status() == 0


def test_release_keeps_to_the_stack():
    cache = kvq.PagedKVCache(1, 2, 1, 64, 16, 4, 8)
    lens, table = ints([64, 40]), ints(np.arange(16).reshape(2, 8) % 4)
    free, count = ints([3, -1, -1, -1]), ints([1])
    cache.release(ints([1, 1]), lens, table, free, count)  # seven pages onto a stack of four
    torch.cuda.synchronize()
    assert count.item() == 4 and lens.tolist() == [0, 0] and free.tolist() == [3, 0, 1, 2]
    with pytest.raises(kvq.KVQError):
        cache.status()
    count = ints([9])
    cache.release(ints([1, 0]), ints([16, 16]), table, free, count)
    torch.cuda.synchronize()
    assert count.item() == 9
    with pytest.raises(kvq.KVQError):
        cache.status()


# -- write and decode --------------------------------------------------------
class Served:
    """A cache with its oracle and the host's view of the tables."""

    def __init__(self, r, h, d, page, code, dtype, longest, layers=1, seed=0):
        self.r, self.h, self.d, self.page, self.code, self.dtype = r, h, d, page, code, dtype
        self.rs = np.random.RandomState(seed)
        self.gen = torch.Generator().manual_seed(seed + 5)
        mp = -(-longest // page)
        self.cache = kvq.PagedKVCache(layers, r, h, d, page, r * mp + 1, mp, CODE[code], dtype)
        self.table = ints(np.full((r, mp), -1))
        self.free = ints(self.rs.permutation(r * mp + 1))
        self.count, self.lens = ints([r * mp + 1]), ints(np.zeros(r))
        self.oracle = PO.PagedOracle(r, h, d, page, code)

    def rows(self, t, heads, spread=1.0):
        x = torch.randn(t, heads, self.d, generator=self.gen)
        return (x * spread).to(self.dtype)

    def step(self, new, layer=0, k=None, v=None, pad=0):
        t = int(np.sum(new)) + pad
        if k is None:
            k, v = self.rows(t, self.h), self.rows(t, self.h)
        plan = self.cache.reserve(self.lens, ints(new), self.table, self.free, self.count, t)
        self.cache.write(layer, k.cuda(), v.cuda(), plan.cu_tokens, plan.slots, plan.lens)
        self.lens, self.count = plan.lens, plan.free_count
        table, at = self.table.cpu().numpy(), 0
        for b, m in enumerate(new):
            self.oracle.write(b, k[at:at + m].double().numpy(), v[at:at + m].double().numpy(), table[b])
            at += m

    def check_state(self):
        pages, scales = self.cache.pages(0).cpu().numpy(), self.cache.scales(0).cpu().numpy()
        tails = self.cache.tails(0).double().cpu().numpy()
        for (p, h, i), c in self.oracle.codes.items():
            assert np.array_equal(pages[p, h, i], c), (p, h, i)
            assert scales[p, h, i] == self.oracle.scales[p, h, i]
        for b in range(self.r):
            x = self.oracle.tail(b).transpose(1, 2, 0, 3)
            assert np.array_equal(tails[b, :, :, :x.shape[2]], x), b

    def check_decode(self, group, scale=None, out_dtype=None, spread=1.0):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        q = self.rows(self.r, self.h * group, spread)
        o = self.cache.decode(0, q.cuda(), self.table, self.lens, scale, out_dtype=out_dtype)
        torch.cuda.synchronize()
        assert o.dtype == (out_dtype or self.dtype)
        got, table = o.double().cpu().numpy(), self.table.cpu().numpy()
        eps = torch.finfo(o.dtype).eps / 2
        for b in range(self.r):
            kv = self.oracle.values(b, table[b])
            for hq in range(self.h * group):
                if kv.shape[2] == 0:
                    assert not got[b, hq].any()
                    continue
                k, v = kv[0, hq // group], kv[1, hq // group]
                ref, w, size = PO.attend(q[b, hq].double().numpy(), k, v, scale)
                err = np.abs(got[b, hq] - ref)
                tol = decode_bound(w, size, np.abs(v).max(), len(v), eps, ref)
                assert (err <= tol).all(), (b, hq, float((err / tol).max()))


STEPS = [[[37, 0, 5, 130], [1, 1, 1, 1], [60, 17, 0, 64], [1, 0, 200, 1], [70, 111, 59, 61]]]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code,dtype", [("int8", F16), ("int8", BF16), ("e4m3", F16), ("e4m3", BF16)])
def test_write_and_decode(page, d, code, dtype):
    """Chunks that start and end anywhere in a page, single tokens, idle slots."""
    s = Served(4, 2, d, page, code, dtype, 512, seed=page + d)
    for i, new in enumerate(STEPS[0]):
        s.step(new, pad=3 * (i % 2))
        s.check_state()
        s.check_decode(group=3)
    assert s.cache.status() == 0


@pytest.mark.parametrize("group", [1, 2, 4, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_head_groups(group, dtype):
    s = Served(3, 2, 128, 32, "e4m3" if group % 2 else "int8", dtype, 256, seed=group)
    s.step([200, 0, 33])
    s.check_decode(group)
    s.check_decode(group, out_dtype=torch.float32)
    s.check_decode(group, scale=-0.05)
    s.check_decode(group, scale=0.0)
    assert s.cache.status() == 0


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 5000])
def test_decode_lengths(n):
    s = Served(2, 1, 64, 64, "int8", F16, 5056, seed=n)
    s.step([n, 0])
    s.check_decode(4)
    s.step([0, n])
    s.check_decode(4, spread=8.0)  # sharp weights: the running maximum moves


def test_decode_many_short_requests_and_few_long_ones():
    """Ranges that hold many requests, and requests cut into many ranges."""
    s = Served(300, 3, 64, 16, "e4m3", BF16, 64, seed=1)
    s.step(s.rs.randint(0, 60, 300))
    s.check_decode(2)
    s = Served(2, 1, 128, 128, "int8", F16, 40064, seed=2)
    s.step([40001, 23456])
    s.check_decode(2)


def test_uneven_values():
    """bf16 rows far outside fp16's range, zero pages, one large channel, a key that wins late."""
    s = Served(2, 1, 128, 32, "int8", BF16, 256, seed=4)
    k, v = s.rows(180, 1), s.rows(180, 1)
    k[:, :, 3] *= 50.0
    v[:40] = 0
    v[40:] = (v[40:].float() * 1e12).to(BF16)
    k[150:] = (k[150:].float() * 6).to(BF16)
    s.step([110, 70], k=k, v=v)
    s.check_state()
    s.check_decode(4, scale=0.02)
    s = Served(1, 1, 64, 16, "e4m3", BF16, 256, seed=5)
    tiny = (s.rows(50, 1).float() * 1e-30).to(BF16)
    s.step([50], k=s.rows(50, 1), v=tiny)
    s.check_state()
    s.check_decode(4)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_nonfinite_rows_stay_with_their_request_and_head(bad, code):
    s = Served(3, 2, 64, 16, code, F16, 64, seed=6)
    k, v = s.rows(90, 2), s.rows(90, 2)
    v[35, 1, 7] = bad   # request 1, head 1, in a page that gets full
    k[85, 0, 2] = bad   # request 2, head 0, in the tail
    s.step([30, 30, 30], k=k, v=v)
    q = s.rows(3, 8).cuda()
    o = s.cache.decode(0, q, s.table, s.lens, 0.1)
    fine = torch.isfinite(o).all(-1).cpu()
    want = torch.ones(3, 8, dtype=torch.bool)
    want[1, 4:] = False
    # a key of +inf scores q * inf: -inf, a weight of exactly 0, where q is negative there
    want[2, :4] = (q[2, :4, 2] < 0).cpu() if bad > 0 else False
    assert torch.equal(fine, want)
    assert torch.isnan(o[1, 4:].float()).all()  # the page reads back as NaN throughout
    # what lies in the open page behind the last token is not read
    s.cache.tails(0)[0, :, :, 30 % 16:] = bad
    assert torch.equal(s.cache.decode(0, q, s.table, s.lens, 0.1)[0], o[0])


def test_bad_pages_slots_and_lengths_set_the_status():
    s = Served(3, 2, 64, 16, "int8", F16, 64, seed=7)
    s.step([40, 20, 30])
    q = s.rows(3, 4).cuda()
    good = s.cache.decode(0, q, s.table, s.lens, 0.1)
    table = s.table.clone()
    table[1, 0] = 1 << 30
    table[2, 1] = -5
    o = s.cache.decode(0, q, table, s.lens, 0.1)
    assert torch.equal(o[0], good[0])
    with pytest.raises(kvq.KVQError):
        s.cache.status()
    o = s.cache.decode(0, q, s.table, ints([40, 20, 1 << 20]), 0.1)
    assert torch.equal(o[:2], good[:2]) and not o[2].any()
    with pytest.raises(kvq.KVQError):
        s.cache.status()
    before = s.cache.buffer[256:].clone()
    k = s.rows(16, 2).cuda()
    cu = ints([0, 0, 0, 16])
    for slots, lens in [(ints(np.full(16, -1)), [40, 20, 32]), (ints(np.full(16, 1 << 30)), [40, 20, 32]),
                        (ints(np.full(16, 3)), [40, 20, 32]), (ints(np.full(16, 15)), [40, 20, 5])]:
        s.cache.write(0, k, k, cu, slots, ints(lens))
        assert torch.equal(s.cache.buffer[256:], before)
        with pytest.raises(kvq.KVQError):
            s.cache.status()
    for bad_cu in ([0, 0, 0, 17], [-3, 0, 0, 13], [5, 0, 0, 0]):
        s.cache.write(0, k, k, ints(bad_cu), ints(np.full(16, -1)), ints([40, 20, 17]))
    assert torch.equal(s.cache.buffer[256:], before)
    with pytest.raises(kvq.KVQError):
        s.cache.status()
    assert torch.equal(s.cache.decode(0, q, s.table, s.lens, 0.1), good)


def test_arguments_are_checked():
    s = Served(2, 2, 64, 16, "int8", F16, 64)
    s.step([5, 9])
    q = s.rows(2, 4).cuda()
    c = s.cache
    for bad in (lambda: c.decode(1, q, s.table, s.lens, 0.1), lambda: c.decode(0, q[:, :3], s.table, s.lens, 0.1),
                lambda: c.decode(0, q, s.table, s.lens, float("nan")),
                lambda: c.decode(0, q, s.table, s.lens, 0.1, out_dtype=BF16),
                lambda: c.decode(0, q, s.table, s.lens, 0.1, workspace=torch.empty(16, device="cuda"))):
        with pytest.raises(kvq.KVQError):
            bad()
    for bad in (lambda: c.decode(0, q.float(), s.table, s.lens, 0.1), lambda: c.decode(0, q, s.table.long(), s.lens, 0.1),
                lambda: c.decode(0, q.cpu(), s.table, s.lens, 0.1),
                lambda: c.decode(0, q, s.table, s.lens, 0.1, workspace=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: c.decode(0, q, s.table[:, :2], s.lens, 0.1), lambda: c.decode(0, q, s.table, s.lens[:1], 0.1),
                lambda: c.decode(0, q.transpose(0, 1), s.table, s.lens, 0.1)):
        with pytest.raises(ValueError):
            bad()
    k, ok = s.rows(4, 2).cuda(), lambda *n: ints(np.zeros(n))
    for bad in (lambda: c.write(1, k, k, ok(3), ok(4), s.lens), lambda: c.write(-1, k, k, ok(3), ok(4), s.lens),
                lambda: c.reserve(ok(3), ok(3), ok(3, 4), ok(9), ok(1), 4),       # more requests than slots
                lambda: c.release(ok(3), ok(3), ok(3, 4), ok(9), ok(1))):
        with pytest.raises(kvq.KVQError):
            bad()
    for bad in (lambda: c.write(0, k, k[:3], ok(3), ok(4), s.lens), lambda: c.write(0, k, k, ok(3), ok(3), s.lens),
                lambda: c.reserve(ok(2), ok(3), ok(2, 4), ok(9), ok(1), 4), lambda: c.reserve(ok(2), ok(2), ok(2, 5), ok(9), ok(1), 4),
                lambda: c.reserve(ok(2), ok(2), ok(2, 4), ok(8), ok(1), 4), lambda: c.reserve(ok(2), ok(2), ok(2, 4), ok(9), ok(1), -1)):
        with pytest.raises(ValueError):
            bad()
    c.write(0, k[:0], k[:0], ok(3), ok(0), s.lens)  # nothing to write
    c.reserve(s.lens, ok(2), s.table, s.free, s.count, 0)
    assert c.status() == 0


def test_layers_and_strided_rows():
    """Layers keep apart; k, v, q as slices of one projection."""
    h, g, d = 2, 4, 128
    cache = kvq.PagedKVCache(3, 2, h, d, 16, 12, 6, kvq.PAGE_INT8, F16)
    table, free = ints(np.full((2, 6), -1)), ints(np.arange(12))
    plan = cache.reserve(ints([0, 0]), ints([50, 21]), table, free, ints([12]), 71)
    outs = []
    for layer in range(3):
        x = torch.randn(71, h * g + 2 * h, d, generator=torch.Generator().manual_seed(layer)).half().cuda()
        k, v = x[:, h * g:h * g + h], x[:, h * g + h:]
        cache.write(layer, k, v, plan.cu_tokens, plan.slots, plan.lens)
        q = x[[49, 70], :h * g]
        outs.append((cache.decode(layer, q, table, plan.lens, 0.09), q, k, v))
    for layer, (o, q, k, v) in enumerate(outs):
        one = kvq.PagedKVCache(1, 2, h, d, 16, 12, 6, kvq.PAGE_INT8, F16)
        one.write(0, k.contiguous(), v.contiguous(), plan.cu_tokens, plan.slots, plan.lens)
        assert torch.equal(one.pages(0), cache.pages(layer)) and torch.equal(one.scales(0), cache.scales(layer))
        assert torch.equal(one.decode(0, q.contiguous(), table, plan.lens, 0.09), o)
        assert torch.equal(cache.decode(layer, q, table, plan.lens, 0.09), o)  # the same bits every time
    assert cache.status() == 0


def test_serving_steps_eager_and_replayed_from_a_graph():
    """Prompts, then decode steps with a finished and an admitted request: the
    eager loop, and the same decode steps as replays of one captured step."""
    r, h, g, d, page = 3, 2, 4, 64, 16
    def serve(graph):
        gen = torch.Generator().manual_seed(9)
        cache = kvq.PagedKVCache(1, r, h, d, page, 40, 12, kvq.PAGE_E4M3, BF16)
        table, free, count, lens = ints(np.full((r, 12), -1)), ints(np.arange(40)), ints([40]), ints([0, 0, 0])
        outs = []
        def admit(new):
            t = int(sum(new))
            x = torch.randn(t, h * g + 2 * h, d, generator=gen).to(BF16).cuda()
            plan = cache.reserve(lens, ints(new), table, free, count, t, lens_out=lens, free_count_out=count)
            k, v = x[:, h * g:h * g + h], x[:, h * g + h:]
            outs.append(kvq.prompt_attention(x[:, :h * g], k, v, plan.cu_tokens, 0.125))
            cache.write(0, k, v, plan.cu_tokens, plan.slots, plan.lens)
        x = torch.zeros(r, h * g + 2 * h, d, dtype=BF16, device="cuda")
        new, out = ints([1, 1, 0]), torch.zeros(r, h * g, d, dtype=BF16, device="cuda")
        ws = torch.empty(cache.workspace_bytes(h * g), dtype=torch.uint8, device="cuda")
        plan = cache.reserve(lens, ints([0, 0, 0]), table, free, count, r, lens_out=lens, free_count_out=count)
        def one():
            cache.reserve(lens, new, table, free, count, r, plan=plan)
            cache.write(0, x[:, h * g:h * g + h], x[:, h * g + h:], plan.cu_tokens, plan.slots, lens)
            cache.decode(0, x[:, :h * g], table, lens, 0.125, out=out, workspace=ws)
        run = one
        if graph:
            keep = [t.clone() for t in (lens, table, free, count, cache.buffer)]
            one()
            torch.cuda.synchronize()
            for t, k in zip((lens, table, free, count, cache.buffer), keep):
                t.copy_(k)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                one()
            run = gr.replay
        admit([37, 16, 0])
        for i in range(40):
            if i == 13:
                cache.release(ints([0, 1, 0]), lens, table, free, count)
                new.copy_(ints([1, 0, 0]))
            if i == 20:
                admit([0, 0, 70])
                new.copy_(ints([1, 0, 1]))
            # packed tokens: the new ones in order of request; queries: by slot
            x.copy_(torch.randn(r, h * g + 2 * h, d, generator=gen).to(BF16))
            run()
            outs.append(out.clone())
        torch.cuda.synchronize()
        assert cache.status() == 0
        assert count.item() + sum(-(-int(n) // page) for n in lens.tolist()) == 40
        return outs, lens.tolist()
    a, la = serve(False)
    b, lb = serve(True)
    assert la == lb == [77, 0, 90] and len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_other_streams_and_two_graphs():
    """Work on a stream of its own; two captured decodes, each with its workspace, replayed together."""
    s = Served(4, 2, 128, 32, "int8", F16, 640, seed=11)
    s.step([600, 33, 0, 257])
    q = [s.rows(4, 8).cuda() for _ in range(2)]
    want = [s.cache.decode(0, x, s.table, s.lens, 0.1) for x in q]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = s.cache.decode(0, q[0], s.table, s.lens, 0.1, stream=side,
                         workspace=torch.empty(s.cache.workspace_bytes(8), dtype=torch.uint8, device="cuda"))
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs, outs, wss = [], [], []
    for x in q:
        wss.append(torch.empty(s.cache.workspace_bytes(8), dtype=torch.uint8, device="cuda"))
        outs.append(torch.zeros_like(want[0]))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s.cache.decode(0, x, s.table, s.lens, 0.1, out=outs[-1], workspace=wss[-1])
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_pages_past_four_gibibytes():
    """A page whose byte offset passes 2^32, and a table that names it."""
    h, d, page = 8, 128, 128
    pages = (1 << 32) // (h * 2 * page * d) + 40
    cache = kvq.PagedKVCache(1, 1, h, d, page, pages, 4)
    table, free = ints([[-1] * 4]), ints(np.zeros(pages))
    free[:3] = ints([5, pages - 1, pages - 2])
    k, v = (torch.randn(300, h, d, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2))
    plan = cache.reserve(ints([0]), ints([300]), table, free, ints([3]), 300)
    cache.write(0, k, v, plan.cu_tokens, plan.slots, plan.lens)
    q = torch.randn(1, h, d, generator=torch.Generator().manual_seed(3)).half().cuda()
    o = cache.decode(0, q, table, plan.lens, 0.1, out_dtype=torch.float32)
    small = kvq.PagedKVCache(1, 1, h, d, page, 4, 4)
    t2 = ints([[-1] * 4])
    p2 = small.reserve(ints([0]), ints([300]), t2, ints(np.arange(4)), ints([4]), 300)
    small.write(0, k, v, p2.cu_tokens, p2.slots, p2.lens)
    assert table.tolist() == [[pages - 2, pages - 1, 5, -1]]
    assert torch.equal(small.decode(0, q, t2, p2.lens, 0.1, out_dtype=torch.float32), o)
    assert cache.status() == 0


def test_many_requests():
    """4096 slots, most of them idle or short: the plan, the write and the decode."""
    r, page = 4096, 16
    rs = np.random.RandomState(5)
    new = rs.randint(0, 3, r)
    new[[3, 4095]] = [700, 90]
    t = int(new.sum())
    pages = int((-(-new // page)).sum())
    cache = kvq.PagedKVCache(1, r, 1, 64, page, pages, 48)
    table, free = ints(np.full((r, 48), -1)), ints(rs.permutation(pages))
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(t, 1, 64, generator=gen).half() for _ in range(2))
    q = torch.randn(r, 2, 64, generator=gen).half()
    lens, count = ints(np.zeros(r)), ints([pages])
    plan = cache.reserve(lens, ints(new), table, free, count, t, lens_out=lens, free_count_out=count)
    cache.write(0, k.cuda(), v.cuda(), plan.cu_tokens, plan.slots, lens)
    o = cache.decode(0, q.cuda(), table, lens, 0.125).double().cpu().numpy()
    assert count.item() == 0 and np.array_equal(lens.cpu().numpy(), new) and cache.status() == 0
    cu, tab = plan.cu_tokens.tolist(), table.cpu().numpy()
    assert not o[new == 0].any()
    for b in list(np.flatnonzero(new)[:20]) + [3, 4095]:
        oracle = PO.PagedOracle(1, 1, 64, page, "int8")
        oracle.write(0, k[cu[b]:cu[b + 1]].double().numpy(), v[cu[b]:cu[b + 1]].double().numpy(), tab[b])
        kv = oracle.values(0, tab[b])
        for h in range(2):
            ref, w, size = PO.attend(q[b, h].double().numpy(), kv[0, 0], kv[1, 0], 0.125)
            tol = decode_bound(w, size, np.abs(kv[1]).max(), int(new[b]), 2.0 ** -11, ref)
            assert (np.abs(o[b, h] - ref) <= tol).all(), b


def test_shared_pages_are_read_by_both():
    """Two requests whose tables name the same complete pages (a shared prefix)."""
    s = Served(2, 2, 128, 32, "e4m3", F16, 256, seed=3)
    s.step([200, 0])
    table = s.table.clone()
    table[1] = table[0]
    lens = ints([192, 192])
    q = s.rows(1, 8).cuda().repeat(2, 1, 1)
    o = s.cache.decode(0, q, table, lens, 0.1)
    assert torch.equal(o[0], o[1]) and o.any()
    assert s.cache.status() == 0


def test_write_takes_the_rows_after_others():
    """cu_tokens that starts inside the packed rows: the ones before it are not read."""
    cache = kvq.PagedKVCache(1, 1, 1, 64, 16, 4, 4)
    x = torch.randn(100, 1, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    x[:60] = float("nan")
    slots = ints(np.concatenate([np.full(60, -1), np.arange(40)]))
    cache.write(0, x, x, ints([60, 100]), slots, ints([40]))
    other = kvq.PagedKVCache(1, 1, 1, 64, 16, 4, 4)
    other.write(0, x[60:], x[60:], ints([0, 40]), ints(np.arange(40)), ints([40]))
    assert torch.equal(cache.buffer, other.buffer) and cache.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_many_small_weights_beside_a_large_one(dtype, d, code):
    """A first token of e^14.125 times the weight of each other one, which hold
    the values: in pages and in the tail their weights keep 11 bits."""
    for t in (3000, 50):  # tokens in pages and a tail, in the tail alone
        s = Served(1, 1, d, 64, code, dtype, 3100)
        k, v = torch.zeros(t, 1, d, dtype=dtype), torch.ones(t, 1, d, dtype=dtype)
        k[0, 0, 0], v[0] = 14.125, 0
        s.step([t], k=k, v=v)
        q = torch.zeros(1, 1, d, dtype=dtype)
        q[0, 0, 0] = 1
        o = s.cache.decode(0, q.cuda(), s.table, s.lens, 1.0, out_dtype=torch.float32).double()
        n = (t - 1) * math.exp(-14.125)
        # half a step of fp16, and what the codes' scales, exponentials and fp32 sums add
        assert ((o - n / (1 + n)).abs() <= (2.0 ** -11 + 2.0 ** -14) * 1.01 * n).all(), t


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,top", [(F16, 61440.0), (BF16, 2.0 ** 55)])
def test_scores_of_any_size(dtype, top, d):
    """Equal scores far past where a last place of theirs is worth a weight."""
    t = 333
    s = Served(1, 1, d, 64, "int8", dtype, 400)
    s.step([t], k=torch.full((t, 1, d), top, dtype=dtype), v=s.rows(t, 1))
    kv = s.oracle.values(0, s.table.cpu().numpy()[0])[1, 0]
    for sign in (1, -1):
        q = torch.full((1, 1, d), sign * top, dtype=dtype)
        o = s.cache.decode(0, q.cuda(), s.table, s.lens, 0.1, out_dtype=torch.float32)[0, 0].double().cpu().numpy()
        assert np.isfinite(o).all()
        # the pages' keys read back as code * scale, within 2^-23 of the tail's:
        # at these sizes one or the other has all the weight
        near = [kv[:t // 64 * 64].mean(0), kv[t // 64 * 64:].mean(0), kv.mean(0)]
        tol = (2.0 ** -11 + 2.0 ** -14) * np.abs(kv).mean(0) * 2
        assert any((np.abs(o - x) <= tol).all() for x in near)
