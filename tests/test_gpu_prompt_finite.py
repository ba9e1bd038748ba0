"""Prompt attention by comparisons that a NaN cannot pass: `within` asks that
every error is at most its bound, which is false of a NaN."""
import math

import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from tests.test_gpu_prompt_attention import BF16, F16, LENS, check, ints, reference, rows

pytestmark = pytest.mark.gpu


def within(err, tol):
    ok = err <= tol
    assert ok.all(), (int((~ok).sum()), float((err / tol).max()))


@pytest.mark.parametrize("lens", [[1], [31], [33], [128], [129], [300], [0, 5, 0, 260, 1], [1000, 17, 333]], ids=str)
@pytest.mark.parametrize("hq,h", [(2, 1), (3, 1), (4, 4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scale_zero_is_the_mean_of_the_values(lens, hq, h, d, dtype):
    """Every weight is 2^0 exactly: what rounds is the fp32 sum of at most n
    values (2^-23 of the magnitudes each), the division and the output."""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = rows(cu[-1], hq, h, d, dtype, seed=cu[-1] + hq).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
    o = kvq.prompt_attention(q, k, v, ints(cu), 0.0)
    ref, w, _ = reference(q, k, v, cu, 0.0)
    half = torch.finfo(dtype).eps / 2
    # an output below the type's normal range rounds by half its smallest step
    step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    within((o.double() - ref).abs(), (max(lens) + 8) * 2.0 ** -23 * w + half * 1.001 * ref.abs() + step / 2)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("part", ["k", "v"])
def test_scale_zero_and_bad_values_of_later_tokens(bad, part):
    """0 * inf is NaN: neither the score nor the value of a later token comes in."""
    x = rows(300, 2, 1, 128, F16, seed=5).cuda()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    want = kvq.prompt_attention(q, k, v, ints([0, 300]), 0.0)
    (k if part == "k" else v)[157, 0, 9] = bad
    got = kvq.prompt_attention(q, k, v, ints([0, 300]), 0.0)
    assert torch.isfinite(want).all() and torch.equal(got[:157], want[:157])
    assert not torch.isfinite(got[157:, :, 9]).any()


def finite(x, hq, h, lens, scale):
    """`check` compares with `err > tol`, which is false of a NaN as well: with
    finite inputs every row of a sequence has to be finite for it to hold."""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    o = check(x, hq, h, cu, scale)
    bad = ~torch.isfinite(o[:cu[-1]]).flatten(1).all(1)
    assert not bad.any(), bad.nonzero().flatten().tolist()[:8]


@pytest.mark.parametrize("lens", LENS + [[2049, 31]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_of_every_length_are_finite(lens, d, dtype):
    finite(rows(sum(lens), 4, 2, d, dtype, seed=sum(lens) + 1), 4, 2, lens, 1 / math.sqrt(d))


@pytest.mark.parametrize("h,g", [(1, 1), (2, 1), (1, 3), (3, 2), (2, 8), (1, 16), (8, 4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_of_every_head_group_are_finite(h, g, d, dtype):
    finite(rows(300, h * g, h, d, dtype, seed=h * g + 1), h * g, h, [170, 130], 1 / math.sqrt(d))


@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-30, 1e-3, 1.0])
@pytest.mark.parametrize("spread", [0.0, 0.3, 8.0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_at_every_scale_are_finite(scale, spread, dtype):
    finite(rows(300, 2, 1, 64, dtype, seed=3, spread=spread), 2, 1, [300], scale)


@pytest.mark.parametrize("flip", [False, True])
def test_rows_of_rising_and_falling_scores_are_finite(flip):
    x = rows(600, 1, 1, 128, F16, seed=5)
    x[:, 0] = 0.5
    x[:, 1] = (torch.arange(600)[:, None] * 0.02 + 0.01 * torch.randn(600, 128, generator=torch.Generator().manual_seed(2))).half()
    if flip:
        x[:, 1] = x[:, 1].flip(0)
    finite(x, 1, 1, [600], 0.1)
