"""Measured cases of the paged 8-bit serving path: page planning, the paged
cache write, decode attention over the paged cache, and prompt attention over
packed sequences.

One serving step plans its pages on the GPU from the request lengths, runs
causal attention over the prompts' own fp16/bf16 keys and values, writes them
into 8-bit pages with one scale per (page, kv-head), and decodes one token per
request from those pages. Each case is one call of one of the four operators.

``own`` false: elementary torch operations in fp32, rounded once at the end.
``own`` true: the calls of this package. ``exact``: the definition in 64 bits.

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
QMAX = {"int8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # page planning: one decode step of a small batch (latency), and the
        # admission of a large prefill batch beside running requests
        dict(name="plan-step-16", op="plan", requests=16, tokens=16, page=64, max_pages=64, longest=4000, kind="step"),
        dict(name="plan-mixed-1024", op="plan", requests=1024, tokens=262144, page=16, max_pages=512, longest=4096,
             kind="mixed"),
        # cache write: one token for each of eight requests (a decode step);
        # a packed ragged prefill chunk; a long prefill of one 8B-shaped layer
        dict(name="write-step-8", op="write", requests=8, tokens=8, kv_heads=8, dim=128, page=64, code="int8",
             dtype="f16", kind="step"),
        dict(name="write-chunk-ragged", op="write", requests=6, tokens=8191, kv_heads=8, dim=128, page=32, code="e4m3",
             dtype="bf16", kind="chunk"),
        dict(name="write-prompt-131072", op="write", requests=4, tokens=131072, kv_heads=8, dim=128, page=64,
             code="int8", dtype="f16", kind="chunk"),
        # decode attention: one short request (latency); a ragged serving batch
        # with idle slots; long contexts at 8 query heads per kv-head; a
        # multi-head layer with 64 channels per head
        dict(name="decode-one-777", op="decode", requests=1, longest=777, q_heads=32, kv_heads=8, dim=128, page=16,
             code="int8", dtype="f16", ragged=False),
        dict(name="decode-ragged-64", op="decode", requests=64, longest=8192, q_heads=32, kv_heads=8, dim=128, page=64,
             code="e4m3", dtype="bf16", ragged=True),
        dict(name="decode-long-16", op="decode", requests=16, longest=131072, q_heads=64, kv_heads=8, dim=128, page=128,
             code="int8", dtype="f16", ragged=True),
        dict(name="decode-mha-d64", op="decode", requests=24, longest=2500, q_heads=32, kv_heads=32, dim=64, page=32,
             code="e4m3", dtype="f16", ragged=True),
        # prompt attention: one short prompt (latency); a packed ragged batch;
        # one long prompt of an 8B-shaped layer
        dict(name="prompt-one-100", op="prompt", seqs=1, tokens=100, q_heads=8, kv_heads=2, dim=128, dtype="f16"),
        dict(name="prompt-ragged-8", op="prompt", seqs=8, tokens=8190, q_heads=32, kv_heads=8, dim=128, dtype="bf16"),
        dict(name="prompt-one-16384", op="prompt", seqs=1, tokens=16384, q_heads=32, kv_heads=8, dim=128, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "decode", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    code, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128])
    if op == "plan":
        r = _log(rng, 1, 1024)
        kind = rng.choice(["step", "mixed"])
        longest = _log(rng, 64, 4096)
        t = r if kind == "step" else _log(rng, r, 262144)
        return dict(op=op, requests=r, tokens=t, page=page, kind=kind, longest=longest,
                    max_pages=(longest + t) // page + 2)
    if op == "write":
        kind = rng.choice(["step", "chunk"])
        r = _log(rng, 1, 256) if kind == "step" else _log(rng, 1, 16)
        return dict(op=op, requests=r, tokens=r if kind == "step" else _log(rng, max(r, 64), 65536),
                    kv_heads=rng.choice([1, 2, 4, 8, 12]), dim=dim, page=page, code=code, dtype=dtype, kind=kind)
    if op == "decode":
        h, g = rng.choice([1, 2, 4, 8, 10]), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        r = _log(rng, 1, 96)
        longest = _log(rng, 1, max(64, min(131072, (16 * 131072 * 8) // (r * h * 2))))
        return dict(op=op, requests=r, longest=longest, q_heads=h * g, kv_heads=h, dim=dim, page=page, code=code,
                    dtype=dtype, ragged=r > 1)
    h, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    t = _log(rng, 1, 12000)
    return dict(op=op, seqs=min(t, _log(rng, 1, 12)), tokens=t, q_heads=h * g, kv_heads=h, dim=dim, dtype=dtype)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _split(rs, total, parts):
    """`parts` positive lengths of uneven size with the given sum."""
    w = np.exp(rs.normal(0.0, 0.6, parts))
    n = np.maximum(1, np.floor(w / w.sum() * (total - parts)).astype(np.int64))
    n[-1] += total - n.sum()
    if n[-1] < 1:
        n = np.full(parts, total // parts, np.int64)
        n[-1] += total - n.sum()
    return n


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _fused_qkv(gen, tokens, hq, h, d, dtype):
    """q, k, v as a model's fused projection gives them: slices of one tensor,
    keys with uneven channel magnitudes."""
    x = torch.randn((tokens, hq + 2 * h, d), generator=gen, device=DEV)
    sigma = torch.exp(0.5 * torch.randn((h, d), generator=gen, device=DEV))
    x[:, hq:hq + h] *= sigma
    x = x.to(dtype)
    return x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]


def _random_pages(gen, n, h, page, d, code):
    """Codes as a normal source gives them, and a scale for each (page, head, tensor)."""
    x = torch.randn((n, h, 2, page, d), generator=gen, device=DEV, dtype=torch.float16)
    if code == "int8":
        codes = (x * 36).round_().clamp_(-127, 127).to(torch.int8)
    else:
        codes = (x * 120).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    unit = 1 / 36 if code == "int8" else 1 / 120
    scales = unit * torch.exp(0.3 * torch.randn((n, h, 2), generator=gen, device=DEV))
    return codes, scales


def _plan_lens(case, rs):
    r, page = case["requests"], case["page"]
    old = rs.randint(0, case["longest"] + 1, r)
    if case["kind"] == "step":
        return old, np.ones(r, np.int64)
    # a prefill batch: some requests idle, some one more token, the rest prompts
    add = np.zeros(r, np.int64)
    busy = rs.permutation(r)[:max(1, (3 * r) // 4)]
    add[busy] = _split(rs, case["tokens"], len(busy)) if case["tokens"] >= len(busy) else 1
    most = case["max_pages"] * page
    old = np.minimum(old, np.maximum(0, most - add))
    add = np.minimum(add, most - old)
    return old, add


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = dict(case=case)
    op = case["op"]
    if op == "plan":
        r, page, mp = case["requests"], case["page"], case["max_pages"]
        old, add = _plan_lens(case, rs)
        used = (old + page - 1) // page
        need = (old + add + page - 1) // page
        pages = int(need.sum()) + 8
        order = rs.permutation(pages)
        table = np.full((r, mp), -1, np.int64)
        at = 0
        for b in range(r):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        free = np.full(pages, -1, np.int64)
        free[:pages - at] = order[at:]
        st.update(lens=_i32(old), new=_i32(add), table=_i32(table), free=_i32(free), free_count=_i32([pages - at]))
        if own:
            import bit_quantized_kv_kvq_gb300 as kvq
            st["cache"] = kvq.PagedKVCache(1, r, 1, 64, page, pages, mp)
        return st
    if op == "prompt":
        lens = _split(rs, case["tokens"], case["seqs"]) if case["seqs"] > 1 else np.array([case["tokens"]])
        q, k, v = _fused_qkv(gen, case["tokens"], case["q_heads"], case["kv_heads"], case["dim"],
                             DTYPES[case["dtype"]])
        st.update(q=q, k=k, v=v, cu=_i32(np.concatenate([[0], np.cumsum(lens)])), longest=int(lens.max()))
        return st
    h, d, page, r = case["kv_heads"], case["dim"], case["page"], case["requests"]
    dtype = DTYPES[case["dtype"]]
    if op == "write":
        if case["kind"] == "step":
            old, add = rs.randint(0, 4 * page, r), np.ones(r, np.int64)
        else:  # chunks of prompts: each starts on a page border, as chunk sizes are multiples of a page
            old = rs.randint(0, 4, r) * page
            add = _split(rs, case["tokens"], r)
        new = old + add
    else:
        n = np.full(r, case["longest"], np.int64)
        if case["ragged"]:
            n = np.maximum(1, np.floor(case["longest"] * rs.uniform(0.02, 1.0, r)).astype(np.int64))
            n[rs.randint(r)] = 0  # a slot without a request
        old = new = n
    need = (new + page - 1) // page
    mp = (5 if op == "write" else 1) + (case["tokens"] if op == "write" else case["longest"]) // page
    pages = 5 * r + case["tokens"] // page + 2 if op == "write" else int(need.sum()) + 2
    order = rs.permutation(pages)
    table = np.full((r, mp), -1, np.int64)
    at = 0
    for b in range(r):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    # one page and one request more than the cache has, where the plain form puts what nobody reads
    codes, scales = _random_pages(gen, pages + 1, h, page, d, case["code"])
    tails = _normal(gen, (r + 1, h, 2, page, d), dtype)
    st.update(lens=_i32(old), table=_i32(table))
    if op == "write":
        _, k, v = _fused_qkv(gen, case["tokens"], 2 * h, h, d, dtype)
        cu = np.concatenate([[0], np.cumsum(add)])
        b = np.repeat(np.arange(r), add)
        pos = old[b] + np.arange(len(b)) - cu[b]
        st.update(k=k, v=v, cu=_i32(cu), after=_i32(new), slots=_i32(table[b, pos // page] * page + pos % page), request=_i32(b),
                  pos=_i32(pos), items=int(case["tokens"]) // page + r)
    else:
        st.update(q=_normal(gen, (r, case["q_heads"], d), dtype), longest=int(new.max()))
    if own:
        import bit_quantized_kv_kvq_gb300 as kvq
        cache = kvq.PagedKVCache(1, r, h, d, page, pages, mp, code=getattr(kvq, "PAGE_" + case["code"].upper()),
                                 dtype=dtype)
        cache.pages(0).copy_(codes[:pages])
        cache.scales(0).copy_(scales[:pages])
        cache.tails(0).copy_(tails[:r])
        st.update(cache=cache)
    else:
        st.update(codes=codes, scales=scales, tails=tails)
    return st


def _scale(case):
    return 1.0 / math.sqrt(case["dim"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _own(st, case, op)
    return {"plan": _plain_plan, "write": _plain_write, "decode": _plain_decode, "prompt": _plain_prompt}[op](st, case)


def _values(pages, case):
    return pages.view(torch.float8_e4m3fn) if case["code"] == "e4m3" else pages


def _own(st, case, op):
    if op == "plan":
        p = st["cache"].reserve(st["lens"], st["new"], st["table"], st["free"], st["free_count"], case["tokens"])
        return dict(table=st["table"], cu=p.cu_tokens, slots=p.slots, positions=p.positions, lens=p.lens,
                    free_count=p.free_count)
    if op == "write":
        c = st["cache"]
        c.write(0, st["k"], st["v"], st["cu"], st["slots"], st["after"])
        return dict(pages=_values(c.pages(0), case), scales=c.scales(0), tails=c.tails(0))
    if op == "decode":
        return st["cache"].decode(0, st["q"], st["table"], st["lens"], _scale(case))
    import bit_quantized_kv_kvq_gb300 as kvq
    return kvq.prompt_attention(st["q"], st["k"], st["v"], st["cu"], _scale(case))


def _plain_plan(st, case):
    page, t, mp = case["page"], case["tokens"], case["max_pages"]
    old, add = st["lens"].long(), st["new"].long()
    new = old + add
    have, need = (old + page - 1) // page, (new + page - 1) // page
    grow = need - have
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu = torch.cat([zero, torch.cumsum(add, 0)])
    first = torch.cumsum(grow, 0) - grow
    free_count = st["free_count"].long()
    ok = (cu[-1] <= t) & (grow.sum() <= free_count[0]) & (need.max() <= mp) & (add.min() >= 0) & (old.min() >= 0)
    j = torch.arange(mp, device=DEV)
    taken = first[:, None] + j - have[:, None]
    page_of = st["free"][(free_count - 1 - taken).clamp_(0, st["free"].numel() - 1)]
    fresh = (j >= have[:, None]) & (j < need[:, None]) & ok
    table = torch.where(fresh, page_of, st["table"])
    i = torch.arange(t, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_(max=len(old) - 1)
    pos = old[b] + i - cu[b]
    slot = table[b, (pos // page).clamp_(max=mp - 1)] * page + pos % page
    live = (i < cu[-1]) & ok
    return dict(table=table, cu=(cu * ok).int(), slots=torch.where(live, slot, -1).int(),
                positions=torch.where(live, pos, -1).int(), lens=torch.where(ok, new, old).int(),
                free_count=(free_count - grow.sum() * ok).int())


def _plain_write(st, case):
    page, r = case["page"], case["requests"]
    codes, scales, tails = st["codes"], st["scales"], st["tails"]
    old, cu = st["lens"].long(), st["cu"].long()
    new = old + cu[1:] - cu[:-1]
    kv = torch.stack([st["k"], st["v"]], 2).float()  # [token][head][K, V][channel]
    # the pages that this call completes
    done = new // page - old // page
    ends = torch.cumsum(done, 0)
    w = torch.arange(st["items"], device=DEV)
    b = torch.searchsorted(ends, w, right=True).clamp_(max=r - 1)
    real = w < ends[-1]
    at = old[b] // page + w - (ends[b] - done[b])
    pos = (at * page)[:, None] + torch.arange(page, device=DEV)
    tok = cu[b][:, None] + pos - old[b][:, None]
    fresh = (pos >= old[b][:, None])[:, :, None, None, None]
    rows = torch.where(fresh, kv[tok.clamp(0, len(kv) - 1)], tails[b].permute(0, 3, 1, 2, 4).float())
    rows = rows.permute(0, 2, 3, 1, 4)  # [item][head][K, V][token][channel]
    top = rows.abs().amax((3, 4))
    s = top / torch.full_like(top, QMAX[case["code"]])  # a tensor: a scalar divisor becomes a product with its reciprocal
    y = torch.where((s > 0)[..., None, None], rows / s[..., None, None], 0.0)
    if case["code"] == "int8":
        c = y.round().clamp_(-127, 127).to(torch.int8)
    else:
        c = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    last = (cu[b] + (at + 1) * page - 1 - old[b]).clamp(0, len(kv) - 1)
    dest = torch.where(real, st["slots"].long()[last] // page, len(codes) - 1)
    codes[dest] = c
    scales[dest] = s
    # the rows of each request's open page
    req, p = st["request"].long(), st["pos"].long()
    open_row = p // page == new[req] // page
    tails[torch.where(open_row, req, r), :, :, p % page] = kv.to(tails.dtype)
    return dict(pages=_values(codes[:-1], case), scales=scales[:-1], tails=tails[:-1])


def _plain_decode(st, case):
    h, d, page, r = case["kv_heads"], case["dim"], case["page"], case["requests"]
    g = case["q_heads"] // h
    lens = st["lens"].long()
    n = -(-st["longest"] // page)
    ids = st["table"].long()[:, :n].clamp(min=0)
    x = _values(st["codes"], case)[ids].float() * st["scales"][ids][..., None, None]  # [r][n][h][2][page][d]
    open_page = (torch.arange(n, device=DEV) == (lens // page)[:, None])[:, :, None, None, None, None]
    x = torch.where(open_page, st["tails"][:r, None].float(), x)
    x = x.permute(0, 2, 3, 1, 4, 5).reshape(r, h, 2, n * page, d)
    seen = torch.arange(n * page, device=DEV) < lens[:, None]
    x = torch.where(seen[:, None, None, :, None], x, 0.0)
    q = st["q"].float().view(r, h, g, d)
    s = torch.matmul(q, x[:, :, 0].transpose(2, 3)) * _scale(case)
    p = torch.softmax(s.masked_fill_(~seen[:, None, None, :], float("-inf")), 3)
    o = torch.matmul(torch.where(seen[:, None, None, :], p, 0.0), x[:, :, 1])
    return o.reshape(r, h * g, d).to(st["q"].dtype)


def _plain_prompt(st, case):
    h, d, t = case["kv_heads"], case["dim"], case["tokens"]
    g, n = case["q_heads"] // h, st["longest"]
    cu = st["cu"].long()
    at = cu[:-1, None] + torch.arange(n, device=DEV)  # a padded batch [sequence][row]
    at = at.clamp_(max=t - 1)
    q = st["q"][at].float().view(-1, n, h, g, d).permute(0, 2, 3, 1, 4)
    k = st["k"][at].float().permute(0, 2, 3, 1)[:, :, None]
    v = st["v"][at].float().permute(0, 2, 1, 3)[:, :, None]
    s = torch.matmul(q, k).mul_(_scale(case))
    i = torch.arange(n, device=DEV)
    p = torch.softmax(s.masked_fill_(i[:, None] < i, float("-inf")), 4)
    del s
    o = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(-1, n, h * g, d).to(st["q"].dtype)
    tok = torch.arange(t, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return o[b, tok - cu[b]]


# --------------------------------------------------------------------------
# what one pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        r, t = case["requests"], case["tokens"]
        grown = t // case["page"] + (0 if case["kind"] == "step" else r)
        return dict(bytes=4 * (4 * r + 2 * t + 2 * grown), flops=0)
    d, h = case["dim"], case["kv_heads"]
    if op == "write":
        rows = case["tokens"] * h * 2
        # a step's row goes to the open page in the input's type; a chunk's rows become codes
        out = 2 * d if case["kind"] == "step" else d + 4 / case["page"]
        return dict(bytes=rows * (2 * d + out), flops=3 * rows * d)
    hq = case["q_heads"]
    if op == "decode":
        # a ragged batch: lengths spread evenly up to the longest, one slot empty
        tokens = case["longest"] * (0.51 * (case["requests"] - 1) if case["ragged"] else case["requests"])
        return dict(bytes=tokens * h * 2 * (d + 4 / case["page"]) + 4 * case["requests"] * hq * d,
                    flops=4 * tokens * hq * d)
    t = case["tokens"]
    pairs = t * t / case["seqs"] / 2 + t / 2
    return dict(bytes=2 * t * d * (2 * hq + 2 * h), flops=4 * pairs * hq * d)


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
    return {"plan": _exact_plan, "write": _exact_write, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](
        st, case)


def _exact_plan(st, case):
    page, t = case["page"], case["tokens"]
    old, add = st["lens"].tolist(), st["new"].tolist()
    table, free = st["table"].cpu().numpy().copy(), st["free"].tolist()
    count = st["free_count"].item()
    cu, slots, positions = [0], [], []
    for b, (n, m) in enumerate(zip(old, add)):
        for p in range(n, n + m):
            if p % page == 0:
                count -= 1
                table[b, p // page] = free[count]
            slots.append(int(table[b, p // page]) * page + p % page)
            positions.append(p)
        cu.append(cu[-1] + m)
    pad = [-1] * (t - len(slots))
    return dict(table=_i32(table), cu=_i32(cu), slots=_i32(slots + pad), positions=_i32(positions + pad),
                lens=_i32(np.array(old) + np.array(add)), free_count=_i32([count]))


def _round_e4m3(y):
    """The nearest value of 1 sign, 4 exponent and 3 fraction bits, ties to even, at most 448."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_write(st, case):
    page, code = case["page"], case["code"]
    codes, scales, tails = st["codes"], st["scales"].double(), st["tails"]
    values = _values(codes, case).clone() if code == "e4m3" else codes.clone()
    old, cu, slots = st["lens"].tolist(), st["cu"].tolist(), st["slots"].tolist()
    for b, n in enumerate(old):
        rows = torch.stack([st["k"][cu[b]:cu[b + 1]], st["v"][cu[b]:cu[b + 1]]]).permute(2, 0, 1, 3)
        head = n - n % page
        x = torch.cat([tails[b, :, :, :n % page], rows], 2)  # [head][K, V][token][channel] from the page border on
        end = n + cu[b + 1] - cu[b]
        for at in range(head, end - page + 1, page):
            y = x[:, :, at - head:at - head + page].double()
            top = y.abs().amax((2, 3), keepdim=True)
            s = (top / QMAX[code]).float().double()  # the stored scale is fp32
            ratio = torch.where(s > 0, (y / s.clamp(min=1e-300)).float().double(), 0.0)
            to = slots[cu[b] + at + page - 1 - n] // page
            if code == "int8":
                values[to] = torch.round(ratio).clamp(-127, 127).to(torch.int8)
            else:
                values[to] = _round_e4m3(ratio).float().to(torch.float8_e4m3fn)
            scales[to] = (top / QMAX[code])[:, :, 0, 0]
        left = end % page
        rest = x[:, :, x.shape[2] - left:] if left else x[:, :, :0]
        tails[b, :, :, :left] = rest
    return dict(pages=values[:-1], scales=scales[:-1], tails=tails[:-1].double())


def _exact_decode(st, case):
    h, d, page, r = case["kv_heads"], case["dim"], case["page"], case["requests"]
    g = case["q_heads"] // h
    out = torch.zeros((r, h, g, d), dtype=torch.float64, device=DEV)
    values = _values(st["codes"], case)
    table = st["table"].long()
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        full, left = n // page, n % page
        ids = table[b, :full]
        x = values[ids].float().double() * st["scales"][ids].double()[..., None, None]
        x = x.permute(1, 2, 0, 3, 4).reshape(h, 2, full * page, d)
        x = torch.cat([x, st["tails"][b, :, :, :left].double()], 2)
        s = torch.einsum("hgd,hnd->hgn", st["q"][b].double().view(h, g, d), x[:, 0]) * _scale(case)
        p = torch.exp(s - s.amax(2, keepdim=True))
        out[b] = torch.einsum("hgn,hnd->hgd", p, x[:, 1]) / p.sum(2, keepdim=True)
    return out.view(r, h * g, d)


def _exact_prompt(st, case):
    h = case["kv_heads"]
    g = case["q_heads"] // h
    cu = st["cu"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for lo, hi in zip(cu[:-1], cu[1:]):
        for head in range(case["q_heads"]):
            k, v = st["k"][lo:hi, head // g].double(), st["v"][lo:hi, head // g].double()
            for a in range(lo, hi, 4096):  # rows in parts: fewer of the masked products
                e = min(hi, a + 4096)
                s = st["q"][a:e, head].double() @ k[:e - lo].T * _scale(case)
                later = torch.arange(e - lo, device=DEV) > torch.arange(a - lo, e - lo, device=DEV)[:, None]
                s = s.masked_fill_(later, float("-inf"))
                p = torch.exp(s - s.amax(1, keepdim=True))
                out[a:e, head] = (p @ v[:e - lo]) / p.sum(1, keepdim=True)
    return out
