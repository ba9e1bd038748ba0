"""State of the paged path that outlives a call: a refused plan changes
nothing, whatever it was refused for; memory belongs to the stream that a call
was given."""
import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from tests.test_gpu_paged import F16, ints

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
