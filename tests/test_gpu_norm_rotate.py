"""Norm and rotation of queries and keys against the oracle in 64 bits."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from oracle import paged_oracle as PO
from tests.test_gpu_paged import BF16, F16, ints

pytestmark = pytest.mark.gpu


def bound(ref, size, dtype, normed):
    """Half a step of the output; fp32: a sine or cosine is off by 2^-22 (the angle's
    2^-25 turns and the function's own), the products and sums round four times; the norm's
    sum over 128 squares, root and products add at most 16 roundings of 2^-24. Below
    the type's normal numbers half a step is absolute."""
    half = 2.0 ** -11 if dtype == F16 else 2.0 ** -8
    return half * np.abs(ref) + (2.0 ** -21 + (2.0 ** -19 if normed else 0)) * size * 1.01 + (2.0 ** -25 if dtype == F16 else 0)


def rows(t, heads, d, dtype, seed, spread=1.0):
    x = torch.randn(t, heads, d, generator=torch.Generator().manual_seed(seed))
    return (x * spread).to(dtype)


def check(out, x, pos, inv_freq, rot, w, eps=1e-6, magnitude=1.0):
    ref, size = PO.rotate(x.double().cpu().numpy(), pos, inv_freq, rot.interleaved, magnitude,
                          None if w is None else w.double().cpu().numpy(), eps)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= bound(ref, size, x.dtype, w is not None)).all()


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 8), (128, 120), (64, 64), (64, 16), (64, 0)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (5, 32, 8), (1100, 5, 3), (33, 7, 7)])
def test_norm_rotate(d, rot, dtype, interleaved, tokens, hq, hk):
    freq = [500000.0 ** (-2 * j / max(rot, 1)) for j in range(rot // 2)]
    r = kvq.Rotation(freq, interleaved=interleaved)
    x = rows(tokens, hq + 2 * hk, d, dtype, tokens + d).cuda()
    q, k = x[:, :hq], x[:, hq:hq + hk]
    pos = np.random.RandomState(d).randint(0, 200000, tokens)
    w = [torch.randn(d, generator=torch.Generator().manual_seed(i)).exp().cuda() for i in range(2)]
    for qw, kw in ((w[0], w[1]), (None, None), (w[0], None)):
        launches = kvq.kernel_launches()
        qo, ko = kvq.norm_rotate(q, k, ints(pos), r, qw, kw, eps=1e-5)
        assert kvq.kernel_launches() == launches + 1
        check(qo, q, pos, freq, r, qw, 1e-5)
        check(ko, k, pos, freq, r, kw, 1e-5)


@pytest.mark.parametrize("theta", [10000.0, 1e6])
def test_far_positions(theta):
    """The last positions that an int32 holds are as exact as the first."""
    r = kvq.Rotation.standard(128, theta=theta)
    freq = [theta ** (-2 * j / 128) for j in range(64)]
    pos = np.array([0, 1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 2, 2 ** 31 - 1])
    q, k = rows(6, 2, 128, F16, 1).cuda(), rows(6, 1, 128, F16, 2).cuda()
    qo, ko = kvq.norm_rotate(q, k, ints(pos), r)
    # 64-bit products of position and frequency: 2^31 * 2^-53 of an angle, far below the bound
    check(qo, q, pos, freq, r, None)
    check(ko, k, pos, freq, r, None)


def test_negative_and_fast_frequencies_and_magnitude():
    freq = [-1.0, 7.0, -1e-3, 3.14159, 0.0, 100.0, -6.5, 1e-9]
    r = kvq.Rotation(freq, magnitude=-1.3)
    q, k = rows(40, 3, 64, BF16, 5).cuda(), rows(40, 3, 64, BF16, 6).cuda()
    pos = np.arange(40) * 977
    qo, ko = kvq.norm_rotate(q, k, ints(pos), r)
    check(qo, q, pos, freq, r, None, magnitude=-1.3)
    check(ko, k, pos, freq, r, None, magnitude=-1.3)
    assert torch.equal(qo[..., 16:], q[..., 16:])  # channels past the pairs


def test_padded_tokens_and_places_of_the_output():
    """Tokens without a position are left; outputs in place, or in a wider tensor."""
    r = kvq.Rotation.standard(128)
    x = rows(70, 6, 128, F16, 3).cuda()
    pos = np.arange(70)
    pos[[0, 33, 69]] = -1
    live = torch.tensor(pos >= 0, device="cuda")
    w = torch.rand(128, device="cuda")
    want_q, want_k = kvq.norm_rotate(x[:, :4], x[:, 4:], ints(pos), r, w, w)
    wide = torch.full((70, 9, 128), 7.0, dtype=F16, device="cuda")
    qo, ko = kvq.norm_rotate(x[:, :4], x[:, 4:], ints(pos), r, w, w, q_out=wide[:, 1:5], k_out=wide[:, 6:8])
    assert torch.equal(qo[live], want_q[live]) and torch.equal(ko[live], want_k[live])
    assert (wide[~live] == 7).all() and (wide[:, [0, 5, 8]] == 7).all()
    y = x.clone()
    kvq.norm_rotate(y[:, :4], y[:, 4:], ints(pos), r, w, w, q_out=y[:, :4], k_out=y[:, 4:])
    assert torch.equal(y[live][:, :4], want_q[live]) and torch.equal(y[live][:, 4:], want_k[live])
    assert torch.equal(y[~live], x[~live])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_of_zeros_and_of_extremes(dtype):
    r = kvq.Rotation.standard(64)
    q = rows(4, 2, 64, dtype, 3).cuda()
    q[0] = 0
    q[1] = torch.finfo(dtype).max if dtype == F16 else 2.0 ** 55
    q[2, 0] *= 2.0 ** -14
    q[3, 1, 7] = float("nan")
    w = torch.ones(64, device="cuda")
    pos = [9, 1, 5, 2]
    k = q.clone()
    qo, ko = kvq.norm_rotate(q, k, ints(pos), r, w, w, eps=1e-6)
    assert torch.equal(qo.nan_to_num(), ko.nan_to_num()) and not qo[0].any()
    assert qo[3, 1].isnan().all() and qo[3, 0].isfinite().all()
    freq = [10000.0 ** (-2 * j / 64) for j in range(32)]
    check(qo[:3], q[:3], pos[:3], freq, r, w)
    # a row without a norm keeps its infinity to its own pair
    q[3, 1, 7] = float("inf")
    qo, _ = kvq.norm_rotate(q, k, ints(pos), r)
    bad = ~qo[3, 1].isfinite()
    assert bad.nonzero().flatten().tolist() == [7, 39]


def test_no_tokens_no_heads_and_streams():
    r = kvq.Rotation.standard(128)
    q, k = rows(3, 2, 128, F16, 1).cuda(), rows(3, 1, 128, F16, 1).cuda()
    want = kvq.norm_rotate(q, k, ints([1, 2, 3]), r)
    qo, ko = kvq.norm_rotate(q[:0], k[:0], ints([]), r)
    assert qo.shape == (0, 2, 128) and ko.shape == (0, 1, 128)
    qo, ko = kvq.norm_rotate(q, k[:, :0], ints([1, 2, 3]), r)
    assert torch.equal(qo, want[0]) and ko.shape == (3, 0, 128)
    pos, side = ints([1, 2, 3]), torch.cuda.Stream()
    torch.cuda.synchronize()
    qo, ko = kvq.norm_rotate(q, k, pos, r, stream=side)
    side.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    gr, a, b = torch.cuda.CUDAGraph(), torch.zeros_like(q), torch.zeros_like(k)
    with torch.cuda.graph(gr):
        kvq.norm_rotate(q, k, pos, r, q_out=a, k_out=b)
    pos.copy_(ints([7, -1, 3]))
    gr.replay()
    want = kvq.norm_rotate(q, k, pos, r)
    assert torch.equal(a[[0, 2]], want[0][[0, 2]]) and torch.equal(b[[0, 2]], want[1][[0, 2]]) and not a[1].any()


def test_refusals():
    r = kvq.Rotation.standard(128)
    q, k, pos = rows(3, 2, 128, F16, 1).cuda(), rows(3, 1, 128, F16, 1).cuda(), ints([0, 1, 2])
    w = torch.ones(128, device="cuda")
    for bad in (lambda: kvq.norm_rotate(q.cpu(), k, pos, r), lambda: kvq.norm_rotate(q, k.bfloat16(), pos, r),
                lambda: kvq.norm_rotate(q.float(), k.float(), pos, r), lambda: kvq.norm_rotate(q, k, pos.long(), r),
                lambda: kvq.norm_rotate(q, k, pos, r, w.half()), lambda: kvq.norm_rotate(q, k, pos, r, w, w.cpu()),
                lambda: kvq.norm_rotate(q, k, pos, kvq.Rotation.standard(128, device="cpu")),
                lambda: kvq.norm_rotate(q, k, pos, r, q_out=torch.zeros_like(q, dtype=BF16))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: kvq.norm_rotate(q, k[:2], pos, r), lambda: kvq.norm_rotate(q, k, pos[:2], r),
                lambda: kvq.norm_rotate(q, k[..., :64], pos, r), lambda: kvq.norm_rotate(q, k, pos, r, w[:64]),
                lambda: kvq.norm_rotate(q[..., ::2], k, pos, r), lambda: kvq.norm_rotate(q, k, pos, r, q_out=q[:2]),
                lambda: kvq.norm_rotate(q, k, pos, r, k_out=q), lambda: kvq.Rotation([1.0, 2.0]),
                lambda: kvq.Rotation([1.0, 2.0, float("inf"), 0.0])):
        with pytest.raises(ValueError):
            bad()
    big = rows(3, 2, 64, F16, 1).cuda()
    for bad in (lambda: kvq.norm_rotate(big, big, pos, r), lambda: kvq.norm_rotate(q, k, pos, r, eps=-1.0),
                lambda: kvq.norm_rotate(q, k, pos, r, eps=float("nan")),
                lambda: kvq.norm_rotate(q, k, pos, kvq.Rotation([0.0] * 4, magnitude=float("inf")))):
        with pytest.raises(kvq.KVQError):
            bad()
