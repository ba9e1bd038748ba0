"""Chunk attention in an fp16 cache whose value scales lie far below fp16's smallest numbers:
such a page's tokens keep their share of the weights, and its values are off by no more than the
output type's own steps."""
import math

import pytest
import torch

from tests.test_gpu_paged import F16, ints
from tests.test_gpu_paged_attend import Filled

pytestmark = pytest.mark.gpu

SMALL = [("int8", k) for k in (-23, -24, -25, -26, -31, -47, -48, -49, -60, -120)] + [
    ("e4m3", k) for k in (-14, -15, -16, -20, -24, -25, -26, -30, -38, -39, -40, -60, -120)]


def close(f, out, q, scale):
    """Rows against the definition in 64 bits. Weights, with the page's factor f in [1/2, 2), are
    rounded to fp16: each is off by 2^-11 of itself, or by 2^-25, which is 2^-24 of a weight
    without its factor, beside a sum of 2^6 or more; the sum is of the same rounded weights, so that
    a token moves the output by its weight's error times its value's distance from the output.
    Scores, exponentials and sums in fp32 as in the other tests. A value scale below fp16's numbers
    rounds the value to 2^-25, times a factor of 1 at most; the output is rounded to 2^-11 of itself or 2^-25."""
    g = f.hq // f.h
    for b, (n, m) in enumerate(zip(f.lens, f.new)):
        lo = int(f.cu[b])
        seen = torch.arange(n, device="cuda") <= n - m + torch.arange(m, device="cuda")[:, None]
        for head in range(f.h):
            k, v = f.kv(b, head)
            for a in range(head * g, (head + 1) * g):
                x = q[lo:lo + m, a].double()
                p = torch.softmax((x @ k.T * scale).masked_fill(~seen, -math.inf), 1)
                ref, w = p @ v, p @ v.abs()
                size = (x.abs() @ k.abs().T * scale).amax(1, keepdim=True)
                tol = (2.0 ** -10 + 2 * 256 * 2.0 ** -23 * size + 2.0 ** -18) * w * 1.01
                tol = tol + n * 2.0 ** -29 * v.abs().amax() + 2.0 ** -11 * ref.abs() + 2.02 * 2.0 ** -25
                err = (out[lo:lo + m, a].double() - ref).abs()
                assert (err <= tol).all(), (b, a, (err / tol).max().item(), err.max().item())


@pytest.mark.parametrize("d,m", [(64, 40), (128, 40), (128, 3)])
@pytest.mark.parametrize("code,k", SMALL)
def test_many_tokens_of_small_pages_beside_a_large_weight(d, m, code, k):
    """One token of 2^16 times the weight of each other one, which together have its share: its
    value is 1.5, theirs are those of a scale of 2^k. As many requests as the GPU has SMs, on the
    same pages, so that blocks are not cut and all of their weights go by the large one's."""
    n, r = 65536 + 16, torch.cuda.get_device_properties(0).multi_processor_count
    f = Filled([n], [m], 4, 1, d, 16, code, F16, seed=7, slots=r)
    c, one = f.cache, f.table[0, 0].item()
    number = (lambda x: int(x)) if code == "int8" else (
        lambda x: torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8).item())
    c.pages(0)[:, :, 0] = 0
    c.pages(0)[one, 0, 0, 0, 0] = number(112)
    c.scales(0)[:, :, 0] = 16 * math.log(2.0) / 112
    c.pages(0)[one, 0, 1] = number(96)
    c.scales(0)[:, :, 1] *= 2.0 ** k / c.scales(0)[:, :, 1].mean()
    c.scales(0)[one, :, 1] = 2.0 ** -6
    q = torch.zeros(m, 4, d, dtype=F16, device="cuda")
    q[..., 0] = 1
    out = c.attend(0, q.repeat(r, 1, 1), ints([m * b for b in range(r + 1)]), f.table.repeat(r, 1), ints([n] * r), 1.0)
    close(f, out[:m], q, 1.0)
    for b in (1, r // 3, r // 2, r - 1):
        close(f, out[b * m:(b + 1) * m], q, 1.0)
    assert c.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code,k", SMALL)
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_pages_of_small_scales(d, code, k, share):
    """Some of the pages, or all, at a scale of 2^k; open rows at its values' size."""
    f = Filled([700, 290], [60, 9], 4, 2, d, 32, code, F16, seed=abs(k))
    gen = torch.Generator(device="cuda").manual_seed(abs(k))
    s = f.cache.scales(0)
    small = torch.rand(s.shape[0], generator=gen, device="cuda") < share
    s[:, :, 1] = torch.where(small[:, None], s[:, :, 1] * 2.0 ** k / s[:, :, 1].mean(), s[:, :, 1])
    if share == 1.0:
        f.cache.tails(0)[:, :, 1] *= 2.0 ** (k + 7)
    close(f, f.attend(), f.q, f.scale)
    assert f.cache.status() == 0


def test_values_that_the_cache_wrote_itself():
    """Subnormal fp16 values, written and attended: as far from the cache's own values as above."""
    import bit_quantized_kv_kvq_gb300 as kvq
    h, d, page, n = 2, 128, 16, 200
    for code, name in ((kvq.PAGE_INT8, "int8"), (kvq.PAGE_E4M3, "e4m3")):
        cache = kvq.PagedKVCache(1, 1, h, d, page, 20, 20, code, F16)
        table, free = ints([[-1] * 20]), ints(list(range(20)))
        plan = cache.reserve(ints([0]), ints([n]), table, free, ints([20]), n)
        gen = torch.Generator().manual_seed(3)
        k, v, q = (torch.randn(n, h, d, generator=gen).half().cuda() for _ in range(3))
        v = (v.float() * torch.logspace(-8, 0, n, device="cuda")[:, None, None]).half()
        cache.write(0, k, v, plan.cu_tokens, plan.slots, plan.lens)
        f = Filled.__new__(Filled)
        f.__dict__.update(cache=cache, hq=h, h=h, d=d, page=page, code=name, dtype=F16, table=table, lens=[n], new=[n], cu=[0, n])
        assert 0 < cache.scales(0)[table[0, 0].item(), :, 1].max().item() < 2.0 ** -24
        close(f, cache.attend(0, q, plan.cu_tokens, table, plan.lens, 0.09), q, 0.09)
        assert cache.status() == 0
