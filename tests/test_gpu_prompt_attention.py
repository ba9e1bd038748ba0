"""Causal attention over packed prompts against fp64, within a bound derived
from its roundings: lengths around the tile borders, head groups, strides,
sequences of no tokens, rows outside every sequence, infinities and NaN."""
import math
import os

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rows(t, hq, h, d, dtype, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, hq + 2 * h, d, generator=gen)
    x[:, :hq] *= spread
    return x.to(dtype)


def reference(q, k, v, cu, scale):
    """(o, sum p |v|, score size) in fp64 on the GPU."""
    g = q.shape[1] // k.shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    w, size = torch.zeros_like(o), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for lo, hi in zip(cu[:-1], cu[1:]):
        if hi <= lo:
            continue
        qs = q[lo:hi].double().transpose(0, 1)
        ks = k[lo:hi].double().transpose(0, 1).repeat_interleave(g, 0)
        vs = v[lo:hi].double().transpose(0, 1).repeat_interleave(g, 0)
        later = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1)
        p = torch.softmax((qs @ ks.transpose(1, 2) * scale).masked_fill(later, float("-inf")), 2)
        o[lo:hi] = (p @ vs).transpose(0, 1)
        w[lo:hi] = (p @ vs.abs()).transpose(0, 1)
        size[lo:hi] = ((qs.abs() @ ks.abs().transpose(1, 2)).masked_fill(later, 0).amax(2) * scale).T
    return o, w, size


def check(x, hq, h, cu, scale, out=None, tokens=None):
    """x: fused rows; the bound: weights rounded to the type (half its eps each,
    or 2^-25 of the row's largest below fp16's normal range), fp32 score sums
    of D products (at most 2 D roundings of 2^-23 on the sum of magnitudes),
    fp32 sums of the weighted values, the output's rounding."""
    x = x.cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
    d = q.shape[2]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = kvq.prompt_attention(q, k, v, ints(cu), scale, out=out, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and o.dtype == x.dtype
    ref, w, size = reference(q, k, v, cu, scale)
    half = torch.finfo(x.dtype).eps / 2
    n = max(hi - lo for lo, hi in zip(cu[:-1], cu[1:]))
    tol = (half * 1.01 + 2 * 2 * d * 2.0 ** -23 * size[..., None] + n * 2.0 ** -23 + 2.0 ** -18) * w
    tol = tol * 1.01 + n * 2.0 ** -25 * float(v.abs().max()) + half * ref.abs()
    err = (o.double() - ref).abs()
    live = torch.zeros(len(x), dtype=torch.bool, device="cuda")
    for lo, hi in zip(cu[:-1], cu[1:]):
        live[lo:hi] = True
    bad = (err > tol)[live]
    assert not bad.any(), (int(bad.sum()), float((err / tol)[live].max()))
    return o


LENS = [[1], [2], [63], [64], [65], [127], [128], [129], [255], [256], [257], [383], [511], [640, 1], [1] * 40,
        [0, 5, 0, 0, 300, 7, 0], [129, 256, 1, 511, 128], [1000, 17, 333]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("d,dtype", [(128, F16), (64, BF16)])
def test_lengths(lens, d, dtype):
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    check(rows(cu[-1], 4, 2, d, dtype, seed=cu[-1]), 4, 2, cu, 1 / math.sqrt(d))


@pytest.mark.parametrize("h,g", [(1, 1), (2, 1), (1, 3), (3, 2), (2, 8), (1, 16), (8, 4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_heads(h, g, d, dtype):
    check(rows(300, h * g, h, d, dtype, seed=h * g), h * g, h, [0, 170, 300], 1 / math.sqrt(d))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_flat_and_sharp_weights(dtype, spread):
    check(rows(700, 2, 1, 128, dtype, seed=3, spread=spread), 2, 1, [0, 700], 1 / math.sqrt(128))


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0])
def test_scales(scale):
    check(rows(300, 2, 1, 64, F16, seed=3, spread=0.3), 2, 1, [0, 300], scale)


def test_rising_scores():
    """Every tile raises the maximum: the sums are rescaled each time."""
    x = rows(600, 1, 1, 128, F16, seed=5)
    x[:, 0] = 0.5
    x[:, 1] = (torch.arange(600)[:, None] * 0.02 + 0.01 * torch.randn(600, 128)).half()
    check(x, 1, 1, [0, 600], 0.1)
    x[:, 1] = x[:, 1].flip(0)
    check(x, 1, 1, [0, 600], 0.1)


def test_a_long_prompt():
    check(rows(5000, 2, 1, 128, BF16, seed=8), 2, 1, [0, 4999, 5000], 1 / math.sqrt(128))
    check(rows(4097, 2, 1, 64, F16, seed=9), 2, 1, [0, 4097], 1 / 8)


def test_rows_outside_every_sequence_are_left():
    x = rows(400, 4, 2, 128, F16, seed=4)
    x[350:] = float("nan")
    x[:3] = float("inf")
    out = torch.full((400, 4, 128), 7.0, dtype=F16, device="cuda")
    kvq.prompt_attention(*(x.cuda()[:, a:b] for a, b in ((0, 4), (4, 6), (6, 8))), ints([3, 3, 200, 350]), 0.1, out=out)
    assert (out[:3] == 7).all() and (out[350:] == 7).all()
    inner = rows(400, 4, 2, 128, F16, seed=4)
    want = check(inner[3:350], 4, 2, [0, 197, 347], 0.1)
    # the same rows elsewhere in the pack: the same results but for the place of the tiles
    assert torch.equal(out[3:350], want)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_later_tokens_do_not_reach_earlier_rows(bad, dtype):
    """A bad value or key at one token leaves the rows before it, the other
    sequences and the other heads bit for bit as they were."""
    cu = [0, 90, 410, 500]
    for at in (91, 150, 217, 218, 345, 409):
        for part in ("k", "v"):
            x = rows(500, 4, 2, 128, dtype, seed=6).cuda()
            q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
            want = kvq.prompt_attention(q, k, v, ints(cu), 0.1)
            (k if part == "k" else v)[at, 1, 5] = bad
            got = kvq.prompt_attention(q, k, v, ints(cu), 0.1)
            assert torch.equal(got[:at], want[:at]) and torch.equal(got[410:], want[410:])
            assert torch.equal(got[:, :2], want[:, :2])
            if part == "v":
                hit = got[at:410, 2:]
                keep = [c for c in range(128) if c != 5]
                assert torch.equal(hit[..., keep], want[at:410, 2:][..., keep])
                b = hit[..., 5].float()
                assert torch.isnan(b).all() if math.isnan(bad) else (b[0] == bad).all() and (b == bad).sum() + torch.isnan(b).sum() == b.numel()


def test_opposite_infinities_give_nan():
    x = rows(200, 1, 1, 64, F16, seed=1)
    x[100, 2, 3], x[120, 2, 3] = float("inf"), float("-inf")
    x = x.cuda()
    o = kvq.prompt_attention(x[:, :1], x[:, 1:2], x[:, 2:], ints([0, 200]), 0.01)[:, 0, 3].float()
    assert torch.isfinite(o[:100]).all() and (o[100:120] == float("inf")).all() and torch.isnan(o[120:]).all()


def test_bad_ranges_set_the_status():
    x = rows(100, 2, 1, 64, F16, seed=2).cuda()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    for cu in ([0, 101], [-5, 50], [0, 40, 2 ** 31 - 1]):
        out = torch.zeros(100, 2, 64, dtype=F16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvq.prompt_attention(q, k, v, ints(cu), 0.1, out=out, status=status)
        assert status.item() != 0
        if len(cu) == 3:
            assert torch.equal(out[:40], kvq.prompt_attention(q[:40], k[:40], v[:40], ints([0, 40]), 0.1))
    # a sequence that ends before it starts holds no rows
    out = torch.zeros(100, 2, 64, dtype=F16, device="cuda")
    kvq.prompt_attention(q, k, v, ints([60, 30, 30]), 0.1, out=out)
    assert not out.any()


def test_stream_graph_and_launch_count():
    x = rows(300, 4, 2, 128, BF16, seed=2).cuda()
    q, k, v, cu = x[:, :4], x[:, 4:6], x[:, 6:], ints([0, 100, 300])
    n = kvq.kernel_launches()
    want = kvq.prompt_attention(q, k, v, cu, 0.1)
    assert kvq.kernel_launches() == n + 1
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = kvq.prompt_attention(q, k, v, cu, 0.1, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kvq.prompt_attention(q, k, v, cu, 0.1, out=out)
    for lens in ([0, 100, 300], [0, 250, 260]):
        cu.copy_(ints(lens))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:lens[2]], kvq.prompt_attention(q, k, v, cu, 0.1)[:lens[2]])


def test_arguments_are_checked():
    x = rows(10, 4, 2, 64, F16, seed=2).cuda()
    q, k, v, cu = x[:, :4], x[:, 4:6], x[:, 6:], ints([0, 10])
    for bad in (lambda: kvq.prompt_attention(q.float(), k, v, cu, 0.1), lambda: kvq.prompt_attention(q, k.bfloat16(), v, cu, 0.1),
                lambda: kvq.prompt_attention(q, k, v, cu.long(), 0.1), lambda: kvq.prompt_attention(q.cpu(), k, v, cu, 0.1)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: kvq.prompt_attention(q, k[:9], v, cu, 0.1), lambda: kvq.prompt_attention(q, k, v[:, :1], cu, 0.1),
                lambda: kvq.prompt_attention(q.transpose(0, 1), k, v, cu, 0.1),
                lambda: kvq.prompt_attention(q, k, v, cu, 0.1, out=torch.empty(10, 4, 32, dtype=F16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: kvq.prompt_attention(q[:, :3], k, v, cu, 0.1), lambda: kvq.prompt_attention(q, k, v, cu, -0.1),
                lambda: kvq.prompt_attention(x[..., :32].contiguous()[:, :4], x[..., :32].contiguous()[:, 4:6],
                                             x[..., :32].contiguous()[:, 6:], cu, 0.1)):
        with pytest.raises(kvq.KVQError):
            bad()


def test_pack_does_not_change_a_sequence():
    """A sequence's rows have the same bits alone, anywhere in a pack, and every time."""
    x = rows(1500, 4, 2, 128, BF16, seed=12).cuda()
    cu = [0, 1, 700, 701, 701, 1100, 1500]
    def run(lo, hi, c):
        y = x[lo:hi]
        return kvq.prompt_attention(y[:, :4], y[:, 4:6], y[:, 6:], ints(c), 0.09)
    whole = run(0, 1500, cu)
    for _ in range(3):
        assert torch.equal(run(0, 1500, cu), whole)
    for lo, hi in zip(cu[:-1], cu[1:]):
        if hi > lo:
            assert torch.equal(run(lo, hi, [0, hi - lo]), whole[lo:hi])


def test_rows_before_the_first_sequence_and_unaligned_output():
    """cu_tokens that starts far in; an output on a 16-byte, not a 32-byte border."""
    x = rows(700, 3, 3, 64, F16, seed=13).cuda()
    q, k, v = x[:, :3], x[:, 3:6], x[:, 6:]
    want = kvq.prompt_attention(q[300:], k[300:], v[300:], ints([0, 150, 400]), 0.125)
    flat = torch.full((700 * 3 * 64 + 8,), 5.0, dtype=F16, device="cuda")
    out = flat[8:].view(700, 3, 64)
    assert out.data_ptr() % 32 == 16
    kvq.prompt_attention(q, k, v, ints([300, 450, 700]), 0.125, out=out)
    assert torch.equal(out[300:], want) and (out[:300] == 5).all() and (flat[:8] == 5).all()


def test_many_sequences():
    lens = np.random.RandomState(3).randint(0, 9, 4096)
    lens[[7, 2000]] = [300, 140]
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = rows(int(cu[-1]), 2, 1, 64, F16, seed=14).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = kvq.prompt_attention(x[:, :2], x[:, 2:3], x[:, 3:], ints(cu), 0.125, status=status)
    assert status.item() == 0
    picks = [0, 1, 7, 8, 1999, 2000, 2001, 4095]
    for s in picks:
        lo, hi = int(cu[s]), int(cu[s + 1])
        if hi > lo:
            y = x[lo:hi]
            assert torch.equal(o[lo:hi], kvq.prompt_attention(y[:, :2], y[:, 2:3], y[:, 3:], ints([0, hi - lo]), 0.125))
    check(x[:int(cu[40])], 2, 1, cu[:41].tolist(), 0.125)


def test_first_call_of_a_process_in_a_capture():
    """Kernels that load while a stream is captured (a fresh process)."""
    import subprocess
    import sys
    code = """
import sys, torch
sys.path.insert(0, %r)
import bit_quantized_kv_kvq_gb300 as kvq
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
x = torch.randn(80, 6, 64, device="cuda").half()
cache = kvq.PagedKVCache(1, 2, 1, 64, 16, 8, 4)
lens, new, table, free, count = i([0, 0]), i([40, 40]), i([[-1] * 4] * 2), i(list(range(8))), i([8])
out = torch.zeros(80, 4, 64, dtype=torch.float16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    plan = cache.reserve(lens, new, table, free, count, 80)
    cache.write(0, x[:, 4:5], x[:, 5:], plan.cu_tokens, plan.slots, plan.lens)
    kvq.prompt_attention(x[:, :4], x[:, 4:5], x[:, 5:], plan.cu_tokens, 0.1, out=out)
    dec = cache.decode(0, x[:2, :4], table, plan.lens, 0.1)
g.replay()
torch.cuda.synchronize()
assert cache.status() == 0 and plan.lens.tolist() == [40, 40] and count.item() == 8 and out.any() and dec.any()
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def near(o, ref, w, dtype, extra=2.0 ** -14):
    """Weights and the output rounded to the type, fp32 sums (extra covers both
    exponentials and sums); no score rounds in the cases that call this."""
    half = torch.finfo(dtype).eps / 2
    err, tol = (o.double() - ref).abs(), (half + extra) * 1.01 * w + half * ref.abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,top", [(F16, 256.0), (F16, 4096.0), (F16, 61440.0), (BF16, 2.0 ** 20), (BF16, 2.0 ** 55)])
def test_scores_of_any_size(dtype, top, d):
    """Scores far past where a last place of theirs is worth a weight: equal
    ones share the output, larger ones take it over."""
    t = 450
    v = torch.randn(t, 1, d, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    q = torch.full((t, 1, d), top, dtype=dtype, device="cuda")
    k = torch.full((t, 1, d), top / 2, dtype=dtype, device="cuda")
    k[[150, 333]] = top
    c = 1 / math.sqrt(d)
    n = torch.arange(1, t + 1, device="cuda").double()[:, None, None]
    mean, size = v.double().cumsum(0) / n, v.double().abs().cumsum(0) / n
    ref, w = mean.clone(), size.clone()
    ref[150:333], w[150:333] = v[150].double(), v[150].double().abs()
    ref[333:] = (v[150].double() + v[333].double()) / 2
    w[333:] = (v[150].double().abs() + v[333].double().abs()) / 2
    near(kvq.prompt_attention(q, k, v, ints([0, t]), c), ref, w, dtype)
    k[:] = top  # lowest scores, all equal
    near(kvq.prompt_attention(-q, k, v, ints([0, t]), c), mean, size, dtype)


@pytest.mark.parametrize("base", [726812.0 - 6000, 726812.0, 726812.0 + 6000, -726816.0, 0.0])
def test_a_raise_among_large_scores(base):
    """Scores (exact sums) that differ by 6 around 2^20 in units of log 2: both
    kinds of token weigh in."""
    t, d = 400, 64
    v = torch.randn(t, 1, d, generator=torch.Generator().manual_seed(7)).half().cuda()
    q = torch.zeros(t, 1, d, dtype=F16, device="cuda")
    k = torch.zeros_like(q)
    q[:, 0, 0], q[:, 0, 1] = 1024, 1
    raw = torch.full((t,), base, dtype=torch.float64, device="cuda")
    raw[[130, 300]] += 6
    raw[390] += 12
    hi = (raw / 1024).floor()
    k[:, 0, 0], k[:, 0, 1] = hi.half(), (raw - 1024 * hi).half()
    assert torch.equal((q.double() * k.double()).sum(2)[:, 0], raw)
    p = torch.softmax((raw[None] - base).expand(t, t).masked_fill(torch.ones(t, t, device="cuda").bool().triu(1), float("-inf")), 1)
    ref = torch.einsum("ij,jhd->ihd", p, v.double())
    w = torch.einsum("ij,jhd->ihd", p, v.double().abs())
    near(kvq.prompt_attention(q, k, v, ints([0, t]), 1.0), ref, w, F16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_small_weights_beside_a_large_one(dtype, d):
    """A first token of e^14.125 times the weight of each other one, which hold
    the values: their weights keep the type's precision."""
    t = 3000
    q = torch.zeros(t, 1, d, dtype=dtype, device="cuda")
    k, v = torch.zeros_like(q), torch.ones_like(q)
    q[:, 0, 0], k[0, 0, 0], v[0] = 1, 14.125, 0
    n = torch.arange(t, device="cuda").double()[:, None, None] * math.exp(-14.125)
    ref = (n / (1 + n)).expand(t, 1, d)
    o = kvq.prompt_attention(q, k, v, ints([0, t]), 1.0)
    # an output below the type's normal range rounds by half its smallest step
    step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    half = torch.finfo(dtype).eps / 2
    assert ((o.double() - ref).abs() <= (2 * half + 2.0 ** -14) * 1.01 * ref + step / 2).all()
