"""Measured cases of serving chunks, drafts and branches over the paged 8-bit
cache: attention of several new tokens per request over all that the cache
holds of it, norm and position rotation of queries and keys, forks of
requests onto shared pages, and the release of such pages.

A step of a server that cuts prompts into chunks, checks drafted tokens or
branches requests: the new queries and keys are normalised and rotated by their
positions, the keys and values written into the cache, and the new tokens of every
request, one or thousands, attend its pages and its open rows, earlier chunks
and shared prefixes included. A fork makes a request that shares the complete
pages of another, and a release gives a page back when its last holder ends.
Each case is one call of one of the four operators.

``own`` false: elementary torch operations, in fp32 but for the angles (64
bits), rounded once at the end. ``own`` true: the calls of this package.
``exact``: the definition in 64 bits.

Layouts (C order): pages [page][kv head][K, V][token][channel] in 8 bits,
scales [page][kv head][K, V] fp32, tails (the rows of each request's open
page) [request][kv head][K, V][token][channel] in the input type, block table
[request][page index] int32.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
THETA, EPS = 500000.0, 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # attention over the cache: a few drafted tokens of each of eight
        # requests (latency)
        dict(name="attend-draft-8", op="attend", kind="draft", requests=8, most=5, longest=1000, q_heads=32, kv_heads=8,
             dim=128, page=16, code="int8", dtype="f16"),
        # a step that mixes chunks of prompts, single tokens and idle slots
        dict(name="attend-mixed-24", op="attend", kind="mixed", requests=24, most=1500, longest=9000, q_heads=32,
             kv_heads=8, dim=128, page=64, code="e4m3", dtype="bf16"),
        # drafts on long contexts at 8 query heads per kv-head: bound by the cache's bytes
        dict(name="attend-draft-long", op="attend", kind="draft", requests=4, most=8, longest=110000, q_heads=64,
             kv_heads=8, dim=128, page=128, code="int8", dtype="bf16"),
        # a late chunk of one long prompt of an 8B-shaped layer: bound by the products
        dict(name="attend-chunk-65536", op="attend", kind="chunk", requests=1, most=2048, longest=65536, q_heads=32,
             kv_heads=8, dim=128, page=64, code="int8", dtype="f16"),
        # a multi-head layer with 64 channels per head, chunks of several prompts
        dict(name="attend-mha-d64", op="attend", kind="chunk", requests=12, most=300, longest=4001, q_heads=16, kv_heads=16,
             dim=64, page=32, code="e4m3", dtype="f16"),
        # norm and rotation: a decode step of sixteen requests (latency); a
        # chunk with neighbouring pairs in half of the channels, no norm; a long prompt
        dict(name="rotate-step-16", op="rotate", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             norm=True, dtype="bf16", longest=131072),
        dict(name="rotate-chunk-4099", op="rotate", tokens=4099, q_heads=12, kv_heads=4, dim=64, rot=32, interleaved=True,
             norm=False, dtype="f16", longest=30000),
        dict(name="rotate-prompt-32768", op="rotate", tokens=32768, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", longest=1 << 20),
        # forks: four requests branch once each; samples of one prompt fill the batch
        dict(name="fork-branch-4", op="fork", requests=8, sources=4, copies=1, longest=700, page=16, kv_heads=2, dim=64,
             layers=2, dtype="f16"),
        dict(name="fork-samples-60", op="fork", requests=64, sources=4, copies=15, longest=16000, page=64, kv_heads=8,
             dim=128, layers=8, dtype="bf16"),
        # release of shared pages: half of eight requests end; a large batch
        # of branches, most of which end
        dict(name="release-8", op="release", requests=8, sources=2, longest=900, page=16, ending=0.5),
        dict(name="release-1024", op="release", requests=1024, sources=60, longest=6000, page=16, ending=0.8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rotate", "fork", "release"])
    page, dim = rng.choice([16, 32, 64, 128]), rng.choice([64, 128])
    code, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["f16", "bf16"])
    if op == "attend":
        kind = rng.choice(["draft", "mixed", "chunk"])
        h, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        r = _log(rng, 1, 32)
        most = rng.randint(2, 12) if kind == "draft" else _log(rng, 13, 2048)
        pairs = 5e8 / (h * g) / r  # query and key pairs of a request, as many as the largest case has of a head
        longest = max(most, _log(rng, max(most, 16), max(most + 16, min(65536, pairs * 2 / most))))
        return dict(op=op, kind=kind, requests=r, most=most, longest=longest, q_heads=h * g, kv_heads=h, dim=dim, page=page,
                    code=code, dtype=dtype)
    if op == "rotate":
        h = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 16000), q_heads=h * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=h, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.7,
                    dtype=dtype, longest=_log(rng, 100, 1 << 20))
    sources = _log(rng, 1, 40)
    if op == "fork":
        copies = _log(rng, 1, max(1, 80 // sources))
        return dict(op=op, requests=sources * (copies + 1) + rng.randint(0, 5), sources=sources, copies=copies,
                    longest=_log(rng, 1, 12000), page=page, kv_heads=rng.choice([1, 2, 4, 8]), dim=dim,
                    layers=rng.choice([1, 2, 4]), dtype=dtype)
    r = max(sources, _log(rng, 1, 1024))
    return dict(op=op, requests=r, sources=sources, longest=_log(rng, 1, max(32, min(30000, 4000000 // r))), page=page,
                ending=rng.choice([0.2, 0.5, 0.9, 1.0]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _random_pages(gen, n, h, page, d, code):
    """Codes as a normal source gives them, and a scale for each (page, head, tensor)."""
    x = torch.randn((n, h, 2, page, d), generator=gen, device=DEV, dtype=torch.float16)
    if code == "int8":
        codes = (x * 36).round_().clamp_(-127, 127).to(torch.int8)
    else:
        codes = (x * 120).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    unit = 1 / 36 if code == "int8" else 1 / 120
    return codes, unit * torch.exp(0.3 * torch.randn((n, h, 2), generator=gen, device=DEV))


def _attend_lens(case, rs):
    """Lengths after the step and new tokens of each request. A step's number
    of tokens is the case's; which request has how many goes by the seed."""
    r, most, longest = case["requests"], case["most"], case["longest"]
    spread = (np.arange(r) + 0.5) / r
    if case["kind"] == "draft":
        new = 1 + np.floor(most * spread).astype(np.int64)
    else:
        new = np.maximum(1, np.floor(most * (0.6 + 0.4 * spread)).astype(np.int64))
        if case["kind"] == "mixed":
            new[:r // 2] = 1  # requests that decode
            new[r // 2:r // 2 + r // 8] = 0  # and some that wait
    new[-1] = most
    new = rs.permutation(new)
    lens = np.maximum(new, np.floor(longest * rs.uniform(0.3, 1.0, r)).astype(np.int64))
    if case["kind"] == "chunk" and r > 1:
        lens[rs.randint(r)] = 0  # a first chunk
    lens = np.maximum(lens, new)
    if r == 1:
        lens[0] = longest
    return lens, new


def _shared_tables(case, rs, sources):
    """Lengths, a table whose row b shares the complete pages of its source's
    prefix, and the number of further holders of each page."""
    r, page = case["requests"], case["page"]
    lens = np.maximum(1, np.floor(case["longest"] * rs.uniform(0.2, 1.0, r)).astype(np.int64))
    source = rs.randint(0, sources, r)
    source[:sources] = np.arange(sources)
    mp = case["longest"] // page + 2
    need = -(-lens // page)
    common = np.minimum(lens, lens[source]) // page  # complete pages of both
    common = np.where(source == np.arange(r), 0, np.floor(common * rs.uniform(0.5, 1.0, r)).astype(np.int64))
    pages = r * (mp - 1) + 5
    order = rs.permutation(pages)
    table, at = np.full((r, mp), -1, np.int64), 0
    for b in range(r):
        table[b, :common[b]] = table[source[b], :common[b]]
        table[b, common[b]:need[b]] = order[at:at + need[b] - common[b]]
        at += need[b] - common[b]
    held = np.zeros(pages, np.int64)
    for b in range(r):
        np.add.at(held, table[b, :need[b]], 1)
    free = np.full(pages, -1, np.int64)
    free[:pages - at] = order[at:]
    return lens, table, np.maximum(held - 1, 0), free, pages - at


def _books(**arrays):
    """Small int32 arrays that a call changes in place, as views of one buffer,
    so that a pass can put all of them back in one copy."""
    parts = {k: np.asarray(v, np.int32) for k, v in arrays.items()}
    buf = _i32(np.concatenate([p.reshape(-1) for p in parts.values()]))
    views, at = {}, 0
    for k, p in parts.items():
        views[k] = buf[at:at + p.size].view(p.shape)
        at += p.size
    return buf, views


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = dict(case=case)
    return {"attend": _prepare_attend, "rotate": _prepare_rotate, "fork": _prepare_fork, "release": _prepare_release}[
        case["op"]](st, case, rs, gen)


def _prepare_attend(st, case, rs, gen):
    r, page, h, d, dtype = case["requests"], case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    lens, new = _attend_lens(case, rs)
    need = -(-lens // page)
    mp, pages = int(need.max()) + 1, int(need.sum()) + 2
    order, at = rs.permutation(pages), 0
    table = np.full((r, mp), -1, np.int64)
    for b in range(r):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    codes, scales = _random_pages(gen, pages, h, page, d, case["code"])
    tails = _normal(gen, (r, h, 2, page, d), dtype)
    # the queries as a slice of a fused projection
    q = _normal(gen, (int(new.sum()), case["q_heads"] + 2 * h, d), dtype)[:, :case["q_heads"]]
    st.update(q=q, table=_i32(table), lens=_i32(lens), cu=_i32(np.concatenate([[0], np.cumsum(new)])),
              host=list(zip(lens.tolist(), new.tolist())))
    if own:
        import bit_quantized_kv_kvq_gb300 as kvq
        cache = kvq.PagedKVCache(1, r, h, d, page, pages, mp, code=getattr(kvq, "PAGE_" + case["code"].upper()), dtype=dtype)
        cache.pages(0).copy_(codes)
        cache.scales(0).copy_(scales)
        cache.tails(0).copy_(tails)
        st.update(cache=cache)
    else:
        st.update(codes=codes, scales=scales, tails=tails)
    return st


def _inv_freq(case):
    rot = case["rot"]
    return [THETA ** (-2.0 * i / rot) for i in range(rot // 2)]


def _prepare_rotate(st, case, rs, gen):
    t, hq, h, d, dtype = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    x = _normal(gen, (t, hq + 2 * h, d), dtype)
    # positions of a packed step: runs that start anywhere
    runs = max(1, min(t, 16))
    lens = np.diff(np.concatenate([[0], np.sort(rs.choice(np.arange(1, t), runs - 1, replace=False)) if runs > 1 else [],
                                   [t]])).astype(np.int64)
    pos = np.concatenate([rs.randint(0, max(1, case["longest"] - n + 1)) + np.arange(n) for n in lens])
    w = torch.exp(0.2 * torch.randn((2, d), generator=gen, device=DEV)) if case["norm"] else None
    st.update(q=x[:, :hq], k=x[:, hq:hq + h], pos=_i32(pos), weights=(w[0], w[1]) if case["norm"] else (None, None))
    if own:
        import bit_quantized_kv_kvq_gb300 as kvq
        st["rotation"] = kvq.Rotation(_inv_freq(case), interleaved=case["interleaved"], device=DEV)
    else:
        st["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=DEV)
    return st


def _prepare_fork(st, case, rs, gen):
    r, page, h, d, n_layers = case["requests"], case["page"], case["kv_heads"], case["dim"], case["layers"]
    sources, copies, dtype = case["sources"], case["copies"], DTYPES[case["dtype"]]
    n = np.maximum(1, np.floor(case["longest"] * rs.uniform(0.3, 1.0, sources)).astype(np.int64))
    slots = rs.permutation(r)
    lens = np.zeros(r, np.int64)
    lens[slots[:sources]] = n
    src = np.repeat(slots[:sources], copies)
    dst = slots[sources:sources * (copies + 1)]
    need, mp = -(-n // page), case["longest"] // page + 2
    pages = sources * (mp - 1) + len(src) + 7
    order, at = rs.permutation(pages), 0
    table = np.full((r, mp), -1, np.int64)
    for i in range(sources):
        table[slots[i], :need[i]] = order[at:at + need[i]]
        at += need[i]
    free = np.full(pages, -1, np.int64)
    free[:pages - at] = order[at:]
    st["books"], views = _books(lens=lens, free_count=[pages - at], shared=np.zeros(pages))
    st["start"] = st["books"].clone()
    st.update(views, table=_i32(table), free=_i32(free), src=_i32(src), dst=_i32(dst))
    tails = [_normal(gen, (r, h, 2, page, d), dtype) for _ in range(n_layers)]
    if own:
        import bit_quantized_kv_kvq_gb300 as kvq
        st["cache"] = kvq.PagedKVCache(n_layers, r, h, d, page, pages, mp, dtype=dtype)
        for i, x in enumerate(tails):
            st["cache"].tails(i).copy_(x)
    else:
        st["tails"] = tails
    return st


def _prepare_release(st, case, rs, gen):
    r = case["requests"]
    lens, table, shared, free, count = _shared_tables(case, rs, min(case["sources"], r))
    done = (rs.uniform(0, 1, r) < case["ending"]).astype(np.int64)
    done[rs.randint(r)] = 1
    st["books"], views = _books(lens=lens, free_count=[count], shared=shared)
    st["start"] = st["books"].clone()
    st.update(views, table=_i32(table), free=_i32(free), done=_i32(done))
    if own:
        import bit_quantized_kv_kvq_gb300 as kvq
        st["cache"] = kvq.PagedKVCache(1, r, 1, 64, case["page"], len(free), table.shape[1])
    return st


def _scale(case):
    return 1.0 / math.sqrt(case["dim"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if op in ("fork", "release"):
        # these change their books in place: each pass starts from the same ones
        st["books"].copy_(st["start"])
    if own:
        return _own(st, case, op)
    return {"attend": _plain_attend, "rotate": _plain_rotate, "fork": _plain_fork, "release": _plain_release}[op](st, case)


def _own(st, case, op):
    if op == "attend":
        return st["cache"].attend(0, st["q"], st["cu"], st["table"], st["lens"], _scale(case))
    if op == "rotate":
        import bit_quantized_kv_kvq_gb300 as kvq
        qw, kw = st["weights"]
        q, k = kvq.norm_rotate(st["q"], st["k"], st["pos"], st["rotation"], q_weight=qw, k_weight=kw, eps=EPS)
        return dict(q=q, k=k)
    c = st["cache"]
    if op == "fork":
        c.fork(st["src"], st["dst"], st["lens"], st["table"], st["free"], st["free_count"], st["shared"])
        return dict(table=st["table"], lens=st["lens"], free_count=st["free_count"], shared=st["shared"],
                    tails=[c.tails(i) for i in range(case["layers"])])
    c.release(st["done"], st["lens"], st["table"], st["free"], st["free_count"], shared=st["shared"])
    return dict(lens=st["lens"], free=st["free"], free_count=st["free_count"], shared=st["shared"])


def _values(codes, case):
    return codes.view(torch.float8_e4m3fn) if case["code"] == "e4m3" else codes


def _plain_attend(st, case):
    h, d, page, hq = case["kv_heads"], case["dim"], case["page"], case["q_heads"]
    g, q = hq // h, st["q"]
    table, at, out = st["table"].long(), 0, []
    values = _values(st["codes"], case)
    for b, (n, m) in enumerate(st["host"]):
        if m == 0:
            continue
        full = n // page
        ids = table[b, :full]
        x = (values[ids].float() * st["scales"][ids][..., None, None]).permute(1, 2, 0, 3, 4).reshape(h, 2, full * page, d)
        x = torch.cat([x, st["tails"][b, :, :, :n - full * page].float()], 2)  # [head][K, V][token][channel]
        rows = q[at:at + m].float().view(m, h, g, d).permute(1, 2, 0, 3).reshape(h, g * m, d)
        s = torch.matmul(rows, x[:, 0].transpose(1, 2)).mul_(_scale(case)).view(h, g, m, n)
        later = torch.arange(n, device=DEV) > torch.arange(n - m, n, device=DEV)[:, None]
        s.masked_fill_(later, float("-inf"))
        s.sub_(s.amax(3, keepdim=True)).exp_()
        norm = s.sum(3, keepdim=True)
        o = torch.matmul(s.view(h, g * m, n), x[:, 1]).view(h, g, m, d) / norm
        out.append(o.permute(2, 0, 1, 3).reshape(m, hq, d).to(q.dtype))
        at += m
        del s
    return torch.cat(out)


def _turn(x, cos, sin, rot, interleaved):
    """Pairs of the first `rot` channels turned by their angles."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rotate(st, case):
    angle = st["pos"].double()[:, None, None] * st["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for name, w in zip("qk", st["weights"]):
        x = st[name].float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        out[name] = _turn(x, cos, sin, case["rot"], case["interleaved"]).to(st[name].dtype)
    return out


def _plain_fork(st, case):
    page, lens, table, shared = case["page"], st["lens"], st["table"], st["shared"]
    src, dst = st["src"].long(), st["dst"].long()
    n = lens[src]
    j = torch.arange(table.shape[1], device=DEV)
    kept = j < (n // page)[:, None]
    opens = (n % page > 0).int()
    k = torch.cumsum(opens, 0) - opens
    new = st["free"][(st["free_count"] - 1 - k).clamp_(min=0).long()]
    rows = torch.where(kept, table[src], table[dst])
    rows = torch.where((j == (n // page)[:, None]) & (opens > 0)[:, None], new[:, None], rows)
    ids = torch.where(kept, table[src], shared.numel())
    shared += torch.bincount(ids.flatten().long(), minlength=shared.numel() + 1)[:-1].int()
    table[dst] = rows
    lens[dst] = n
    st["free_count"] -= opens.sum().int()
    live = (torch.arange(page, device=DEV) < (n % page)[:, None])[:, None, None, :, None]
    for x in st["tails"]:
        x[dst] = torch.where(live, x[src], x[dst])
    return dict(table=table, lens=lens, free_count=st["free_count"], shared=shared, tails=st["tails"])


def _plain_release(st, case):
    page, lens, table, shared, free = case["page"], st["lens"], st["table"], st["shared"], st["free"]
    n = shared.numel()
    gone = st["done"] != 0
    ends = (torch.arange(table.shape[1], device=DEV) < ((lens + page - 1) // page)[:, None]) & gone[:, None]
    ids = torch.where(ends, table, n).flatten().long()
    k = torch.arange(ids.numel(), device=DEV)
    released = torch.bincount(ids, minlength=n + 1)[:-1].int()
    last = torch.full((n + 1,), -1, dtype=torch.long, device=DEV).scatter_reduce_(0, ids, k, "amax")
    freed = torch.cat([released > shared, torch.zeros(1, dtype=torch.bool, device=DEV)])  # nobody holds it any more
    push = freed[ids] & (last[ids] == k)
    place = st["free_count"] + torch.cumsum(push, 0) - 1
    padded = torch.cat([free, free[:1]])
    padded[torch.where(push, place, n)] = torch.where(push, ids, 0).int()
    free.copy_(padded[:-1])
    st["free_count"] += push.sum().int()
    shared.sub_(released).clamp_(min=0)
    lens.masked_fill_(gone, 0)
    return dict(lens=lens, free=free, free_count=st["free_count"], shared=shared)


# --------------------------------------------------------------------------
# what one pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "attend":
        r, most, d, h, hq = case["requests"], case["most"], case["dim"], case["kv_heads"], case["q_heads"]
        # as the lengths are drawn, on average
        n = case["longest"] * (0.65 if r > 1 else 1.0)
        share = {"draft": 0.5, "mixed": 0.3, "chunk": 0.8}[case["kind"]] if r > 1 else 1.0
        m = max(1.0, share * most)
        n = max(n, m)
        return dict(bytes=r * (n * h * 2 * (d + 4 / case["page"]) + 4 * m * hq * d),
                    flops=4 * r * m * (n - m / 2) * hq * d)
    if op == "rotate":
        t, rows = case["tokens"], case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return dict(bytes=4 * rows * case["dim"] + 4 * t, flops=rows * (3 * case["rot"] + (4 * case["dim"] if case["norm"] else 0)))
    if op == "fork":
        pairs = case["sources"] * case["copies"]
        entries = 0.65 * case["longest"] / case["page"]
        # the open rows of each new request in every layer; its table row and the counts
        return dict(bytes=pairs * (case["layers"] * case["kv_heads"] * 4 * case["page"] * case["dim"] + 16 * entries), flops=0)
    entries = case["requests"] * case["ending"] * (0.6 * case["longest"] / case["page"] + 1)
    return dict(bytes=12 * entries + 8 * case["requests"], flops=0)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return {"attend": _exact_attend, "rotate": _exact_rotate, "fork": _exact_fork, "release": _exact_release}[case["op"]](
        st, case)


def _exact_attend(st, case):
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["q_heads"] // h
    cu = st["cu"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    values = _values(st["codes"], case)
    for b, n in enumerate(st["lens"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        left = n % page
        ids = st["table"][b, :n // page].long()
        for head in range(h):
            kv = []
            for i in range(2):
                x = values[ids, head, i].float().double() * st["scales"][ids, head, i].double()[:, None, None]
                kv.append(torch.cat([x.reshape(-1, d), st["tails"][b, head, i, :left].double()]))
            for a in range(head * g, (head + 1) * g):
                s = st["q"][lo:hi, a].double() @ kv[0].T * _scale(case)
                seen = torch.arange(n, device=DEV) <= (n - (hi - lo)) + torch.arange(hi - lo, device=DEV)[:, None]
                p = torch.where(seen, torch.exp(s - torch.where(seen, s, -math.inf).amax(1, keepdim=True)), 0.0)
                out[lo:hi, a] = (p @ kv[1]) / p.sum(1, keepdim=True)
    return out


def _exact_rotate(st, case):
    rot, freq = case["rot"], np.array(_inv_freq(case))
    a = np.outer(st["pos"].cpu().numpy().astype(np.float64), freq)
    turn = torch.tensor(np.exp(1j * a), device=DEV)[:, None]  # as a rotation of the complex plane
    out = {}
    for name, w in zip("qk", st["weights"]):
        x = st[name].double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_fork(st, case):
    page = case["page"]
    lens, table, shared = st["lens"].tolist(), st["table"].cpu().numpy().copy(), st["shared"].tolist()
    free, count = st["free"].tolist(), st["free_count"].item()
    tails = [x.clone() for x in st["tails"]]
    before = list(lens)
    for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
        n = before[s]
        for j in range(n // page):
            table[t, j] = table[s, j]
            shared[table[s, j]] += 1
        if n % page:
            count -= 1
            table[t, n // page] = free[count]
            for x in tails:
                x[t, :, :, :n % page] = x[s, :, :, :n % page]
        lens[t] = n
    return dict(table=_i32(table), lens=_i32(lens), free_count=_i32([count]), shared=_i32(shared),
                tails=[x.double() for x in tails])


def _exact_release(st, case):
    page = case["page"]
    lens, table, shared = st["lens"].tolist(), st["table"].cpu().numpy(), st["shared"].tolist()
    free, count = st["free"].tolist(), st["free_count"].item()
    held = [x + 1 for x in shared]
    freed = []  # in the order of each page's last release
    for b, gone in enumerate(st["done"].tolist()):
        if not gone:
            continue
        for p in table[b, :-(-lens[b] // page)].tolist():
            held[p] -= 1
            if held[p] == 0:
                freed.append(p)
        lens[b] = 0
    free[count:count + len(freed)] = freed
    return dict(lens=_i32(lens), free=_i32(free), free_count=_i32([count + len(freed)]),
                shared=_i32([max(0, x - 1) for x in held]))
