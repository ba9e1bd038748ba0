"""Decode over pages and tail at the ends of the input types' ranges, against fp64."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import BF16, F16, PO, Served, decode_bound

pytestmark = pytest.mark.gpu


def compare(s, q, scale, group):
    o = s.cache.decode(0, q.cuda(), s.table, s.lens, scale, out_dtype=torch.float32).double().cpu().numpy()
    table = s.table.cpu().numpy()
    for b in range(s.r):
        kv = s.oracle.values(b, table[b])
        for hq in range(s.h * group):
            k, v = kv[0, hq // group], kv[1, hq // group]
            ref, w, size = PO.attend(q[b, hq].double().numpy(), k, v, scale)
            tol = decode_bound(w, size, np.abs(v).max(), len(v), 2.0 ** -24, ref)
            assert (np.abs(o[b, hq] - ref) <= tol).all(), (b, hq, float((np.abs(o[b, hq] - ref) / tol).max()))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", [-80, -87, -95, -105, -115, -122, 60, 100])
def test_small_and_large_bf16_queries(exponent, d, code):
    """Queries of 2^exponent against keys of the inverse size: the products with
    the codes are fp16, the scores are of ordinary size."""
    s = Served(2, 2, d, 32, code, BF16, 400, seed=exponent + 200)
    t = 333 + 40
    k = (s.rows(t, 2).float() * 2.0 ** -exponent).to(BF16)
    s.step([333, 40], k=k, v=s.rows(t, 2))
    q = (s.rows(2, 4).float() * 2.0 ** exponent).to(BF16)
    compare(s, q, 0.5, 2)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30, 2.0])
def test_any_finite_scale(scale, dtype):
    s = Served(2, 1, 64, 16, "int8", dtype, 200, seed=4)
    s.step([190, 7])
    compare(s, s.rows(2, 3), scale, 3)
