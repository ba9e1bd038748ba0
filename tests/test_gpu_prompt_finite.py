"""Prompt attention by comparisons that a NaN cannot pass: `within` asks that
every error is at most its bound, which is false of a NaN."""
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from tests.test_gpu_prompt_attention import BF16, F16, ints, reference, rows

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
