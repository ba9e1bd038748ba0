"""State of the paged path that outlives a call: a refused plan changes
nothing, whatever it was refused for; memory belongs to the stream that a call
was given."""
import re

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from bit_quantized_kv_kvq_gb300 import paged
from tests.test_gpu_paged import F16, PO, Served, ints

pytestmark = pytest.mark.gpu


# -- planning ----------------------------------------------------------------
def plan_inputs(r, page, tokens, seed):
    """Lengths, new tokens, table and free stack of a step that fits."""
    rs = np.random.RandomState(seed)
    lens, new = rs.randint(0, 3 * page, r), rs.multinomial(tokens, np.ones(r) / r)
    lens[0], new[0] = page + 1, max(1, new[0])  # an open page that takes tokens
    mp = int((lens + new).max()) // page + 2
    used = -(-lens // page)
    need = -(-(lens + new) // page)
    pages = int(need.sum()) + 5
    order, at = rs.permutation(pages), 0
    table = np.full((r, mp), -1, np.int32)
    for b in range(r):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    free = np.full(pages, -1, np.int32)
    free[:pages - at] = order[at:]
    return lens, new, table, free, pages - at, int((need - used).sum()), mp, pages


@pytest.mark.parametrize("r,page,tokens", [(3, 16, 100), (40, 16, 4000), (40, 16, 30000), (700, 16, 60000)])
@pytest.mark.parametrize("value", [-1, "pages", 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("where", ["first", "last", "open"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_bad_page_refuses_the_whole_step(r, page, tokens, value, where, in_place):
    """One launch and two: the entries popped first and last, and a row's open page."""
    lens, new, table, free, count, grow, mp, pages = plan_inputs(r, page, tokens, r + tokens)
    t = int(new.sum())
    assert 0 < grow <= count
    bad = pages if value == "pages" else value
    if where == "open":
        table[0, 1] = bad
    else:
        free[count - 1 if where == "first" else count - grow] = bad
    cache = kvq.PagedKVCache(1, r, 1, 64, page, pages, mp)
    dl, dt, df, dc = ints(lens), ints(table), ints(free), ints([count])
    kw = dict(lens_out=dl, free_count_out=dc) if in_place else {}
    plan = cache.reserve(dl, ints(new), dt, df, dc, t, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(df.cpu().numpy(), free)
    assert np.array_equal(plan.lens.cpu().numpy(), lens) and plan.free_count.item() == count
    assert not plan.cu_tokens.any() and (plan.slots == -1).all() and (plan.positions == -1).all()
    with pytest.raises(kvq.KVQError) as e:
        cache.status()
    assert e.value.status == 7
    # nothing is written by such a plan
    before = cache.buffer.clone()
    x = torch.ones(t, 1, 64, dtype=F16, device="cuda")
    cache.write(0, x, x, plan.cu_tokens, plan.slots, plan.lens)
    assert torch.equal(cache.buffer, before) and cache.status() == 0


@pytest.mark.parametrize("tokens", [200, 9000])
def test_bad_entries_that_a_step_does_not_take_are_left(tokens):
    """Entries below those popped, and open pages of requests without new tokens."""
    lens, new, table, free, count, grow, mp, pages = plan_inputs(20, 16, tokens, tokens)
    lens[3], new[3], table[3, :2] = 20, 0, -9
    grow = int((-(-(lens + new) // 16) - -(-lens // 16)).sum())
    free[:count - grow] = -9
    assert grow < count
    cache = kvq.PagedKVCache(1, 20, 1, 64, 16, pages, mp)
    dt = ints(table)
    plan = cache.reserve(ints(lens), ints(new), dt, ints(free), ints([count]), int(new.sum()))
    assert np.array_equal(plan.lens.cpu().numpy(), lens + new) and plan.free_count.item() == count - grow
    assert (plan.slots >= 0).all() and cache.status() == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("r,tokens", [(50, 3000), (50, 9000), (3000, 40000)])
def test_steps_in_place_one_after_the_other(r, tokens, graph):
    """Lengths and free count are read and written by the same launches (one,
    or two that overlap), step after step without a wait between them."""
    page, steps = 16, 6
    rs = np.random.RandomState(r)
    new = rs.multinomial(tokens, np.ones(r) / r)
    new[rs.randint(r)] = 0
    t = int(new.sum())
    mp = steps * (int(new.max()) // page + 1) + 1
    pages = steps * (t // page + r)
    order = rs.permutation(pages)
    cache = kvq.PagedKVCache(1, r, 1, 64, page, pages, mp)
    lens, dn, table, free, count = ints(np.zeros(r)), ints(new), ints(np.full((r, mp), -1)), ints(order), ints([pages])
    plan = cache.reserve(lens, ints(np.zeros(r)), table, free, count, t, lens_out=lens, free_count_out=count)
    def run():
        cache.reserve(lens, dn, table, free, count, t, plan=plan)
    if graph:
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            run()
        run = gr.replay
    for _ in range(steps):
        run()
    torch.cuda.synchronize()
    want = (np.full((r, mp), -1, np.int32), None, None, None, np.zeros(r, np.int32), pages)
    for _ in range(steps):
        want = PO.reserve(want[4], new, want[0], order, want[5], t, page)
    for got, ref in zip((table, plan.cu_tokens, plan.slots, plan.positions, lens, count), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref)), ref)
    assert cache.status() == 0


# -- streams -----------------------------------------------------------------
def test_a_cache_on_a_stream_takes_no_memory_of_the_current_one():
    """A block that the current stream's queued work still writes is free for
    that stream's next tensor, not for a cache that another stream zeroes."""
    side = torch.cuda.Stream()
    args = (2, 3, 2, 64, 16, 4000, 8)
    n = kvq.PagedKVCache(*args).nbytes
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = torch.empty(n, dtype=torch.uint8, device="cuda")
    block = late.data_ptr()
    del late
    cache = kvq.PagedKVCache(*args, stream=side)
    side.synchronize()
    lo = cache.buffer.data_ptr()
    assert lo + n <= block or block + n <= lo
    del cache
    # the same with work under way: its late writes stay out of the cache
    late = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(50_000_000)
    late.fill_(255)
    del late
    cache = kvq.PagedKVCache(*args, stream=side)
    torch.cuda.synchronize()
    assert not cache.buffer.any() and cache.status() == 0


class Recorder:
    """The library with the workspace of every decode noted."""

    def __init__(self, lib):
        self.lib, self.ws = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name != "kvq_paged_decode_attention":
            return f
        def call(*args):
            self.ws.append((args[11], args[11] + args[12]))
            return f(*args)
        return call


def apart(ranges):
    ranges = sorted(ranges)
    return all(a[1] <= b[0] for a, b in zip(ranges, ranges[1:]))


def capture(side, call):
    """A graph of one call on `side`, made while another stream is current."""
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gr.capture_begin(capture_error_mode="thread_local")
    try:
        call()
    finally:
        with torch.cuda.stream(side):
            gr.capture_end()
    return gr


def test_workspaces_are_a_streams_or_a_graphs_own(monkeypatch):
    """Without `workspace`: eager calls of two streams and graphs captured on
    a stream that is not the current one, none of which share it."""
    s = Served(4, 2, 128, 32, "int8", F16, 640, seed=11)
    s.step([600, 33, 0, 257])
    q = [s.rows(4, 8).cuda() for _ in range(4)]
    want = [s.cache.decode(0, x, s.table, s.lens, 0.1) for x in q]
    rec = Recorder(paged._lib)
    monkeypatch.setattr(paged, "_lib", rec)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want[0]) for _ in q]
    torch.cuda.synchronize()
    for i, st in ((0, side), (1, other)):
        s.cache.decode(0, q[i], s.table, s.lens, 0.1, out=outs[i], stream=st)
    graphs = [capture(side, lambda i=i: s.cache.decode(0, q[i], s.table, s.lens, 0.1, out=outs[i], stream=side))
              for i in (2, 3)]
    assert len(rec.ws) == 4 and apart(rec.ws)
    # all four at once
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(30):
        for i, st in ((0, side), (1, other)):
            s.cache.decode(0, q[i], s.table, s.lens, 0.1, out=outs[i], stream=st)
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert rec.ws[4:] == rec.ws[:2] * 30  # a stream keeps its own
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert s.cache.status() == 0


def test_graphs_of_the_current_stream_have_workspaces_of_their_own(monkeypatch):
    s = Served(3, 1, 64, 16, "e4m3", F16, 320, seed=2)
    s.step([300, 10, 77])
    q = [s.rows(3, 4).cuda() for _ in range(2)]
    want = [s.cache.decode(0, x, s.table, s.lens, 0.1) for x in q]
    rec = Recorder(paged._lib)
    monkeypatch.setattr(paged, "_lib", rec)
    outs, graphs = [torch.zeros_like(want[0]) for _ in q], []
    for x, o in zip(q, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s.cache.decode(0, x, s.table, s.lens, 0.1, out=o)
        graphs.append(gr)
    assert len(rec.ws) == 2 and apart(rec.ws)
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(30):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want)) and s.cache.status() == 0


# -- status ------------------------------------------------------------------
def test_prompt_attention_reports_through_the_caches_status():
    """As the module's step has it: a bad range is left out, and status() raises."""
    assert re.search(r"prompt_attention\(.*status=cache.status_word", paged.__doc__)
    cache = kvq.PagedKVCache(1, 2, 1, 64, 16, 8, 4)
    x = torch.randn(60, 4, 64, device="cuda").half()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    cu, out = ints([0, 20, 60]), torch.zeros(60, 2, 64, dtype=F16, device="cuda")
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        kvq.prompt_attention(q, k, v, cu, 0.1, out=out, status=cache.status_word)
    def eager():
        kvq.prompt_attention(q, k, v, cu, 0.1, out=out, status=cache.status_word)
    for run in (eager, gr.replay):
        cu.copy_(ints([0, 20, 60]))
        run()
        assert cache.status() == 0 and out.any()
        cu.copy_(ints([0, 20, 61]))
        out[20:] = 7
        run()
        with pytest.raises(kvq.KVQError) as e:
            cache.status()
        assert e.value.status == 7 and (out[20:] == 7).all() and cache.status() == 0
    assert cache.status_word.shape == (1,) and cache.status_word.data_ptr() == cache.buffer.data_ptr()
