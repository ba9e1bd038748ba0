"""Host-only checks of the entry points of chunk attention, rotation, forks and
shared releases, and pins of their oracles."""
import ctypes

import numpy as np
import pytest

import bit_quantized_kv_kvq_gb300 as kvq
from oracle import paged_oracle as PO


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kvq.lib()


def test_null_handles_are_rejected(lib):
    n = ctypes.c_size_t()
    assert lib.kvq_paged_attention_workspace_bytes(None, 4, ctypes.byref(n)) == 1
    assert lib.kvq_paged_attention(None, 0, 1, None, 512, 1, 4, None, None, None, 1.0, None, None, 0, None) == 1
    assert lib.kvq_paged_fork(None, 1, 1, *[None] * 8) == 1
    assert lib.kvq_paged_release_shared(None, 1, *[None] * 7) == 1
    assert lib.kvq_last_error()


def rotate(lib, **kw):
    a = dict(q=0x10000, k=0x20000, qs=1024, ks=256, t=3, hq=8, hk=2, d=128, dtype=1, pos=0x30000, turns=0x40000, rot=128,
             inter=0, mag=1.0, qw=None, kw=None, eps=1e-6, qo=0x50000, ko=0x60000, qos=1024, kos=256)
    a.update(kw)
    return lib.kvq_norm_rotate(a["q"], a["k"], a["qs"], a["ks"], a["t"], a["hq"], a["hk"], a["d"], a["dtype"], a["pos"],
                               a["turns"], a["rot"], a["inter"], a["mag"], a["qw"], a["kw"], a["eps"], a["qo"], a["ko"],
                               a["qos"], a["kos"], None)


ROTATE_BAD = [(dict(q=None), 1), (dict(k=0x20008), 1), (dict(qs=1020), 1), (dict(qs=1016), 1), (dict(ks=248), 1),
              (dict(t=-1), 1), (dict(hq=-1), 1), (dict(hk=70000), 1), (dict(d=96), 2), (dict(dtype=0), 1), (dict(pos=None), 1),
              (dict(pos=0x30002), 1), (dict(turns=None), 1), (dict(turns=0x40004), 1), (dict(rot=4), 1), (dict(rot=136), 1),
              (dict(rot=-8), 1), (dict(mag=float("nan")), 1), (dict(mag=float("inf")), 1), (dict(eps=-1e-6), 1),
              (dict(eps=float("nan")), 1), (dict(qw=0x70004), 1), (dict(kw=0x70008), 1), (dict(qo=None), 1),
              (dict(ko=0x60004), 1), (dict(kos=248), 1), (dict(qos=1 << 40), 1), (dict(qo=0x10000, qos=2048), 1),
              (dict(ko=0x20000, kos=512), 1)]


@pytest.mark.parametrize("kw,status", ROTATE_BAD, ids=[str(b[0]) for b in ROTATE_BAD])
def test_rotation_refusals(lib, kw, status):
    before = kvq.kernel_launches()
    assert rotate(lib, **kw) == status
    assert kvq.kernel_launches() == before


def test_rotation_of_nothing(lib):
    assert rotate(lib, t=0) == 0 and rotate(lib, hq=0, hk=0) == 0


def test_turns_are_the_frequencies():
    r = kvq.Rotation([1.0, -1.0, 6.283185307179586, 0.0], device="cpu")
    t = [x % 2 ** 64 for x in r.turns.tolist()]
    assert t[0] == round(2 ** 64 * 0.15915494309189533576888) or abs(t[0] / 2 ** 64 - 0.15915494309189535) < 1e-16
    assert t[1] == 2 ** 64 - t[0] and t[3] == 0
    assert min(t[2], 2 ** 64 - t[2]) < 2 ** 64 * 1e-15  # once round
    assert kvq.Rotation.standard(64, theta=1e4, device="cpu").dim == 64


# -- pins of the oracle ------------------------------------------------------
def test_oracle_fork_and_shared_release_by_hand():
    table = np.array([[3, 4, 5, -1], [-1] * 4, [-1] * 4], np.int32)
    lens, free, shared = np.array([9, 0, 0]), np.array([0, 1, 2, -1, -1, -1]), np.zeros(6, np.int32)
    lens, table, count, shared = PO.fork(np.array([0, 0]), np.array([2, 1]), lens, table, free, 3, shared, 4)
    assert table.tolist() == [[3, 4, 5, -1], [3, 4, 1, -1], [3, 4, 2, -1]] and count == 1
    assert lens.tolist() == [9, 9, 9] and shared.tolist() == [0, 0, 0, 2, 2, 0]
    assert PO.fork(np.array([0]), np.array([1]), lens, table, free, 1, shared, 4) is None
    lens, free, count, shared = PO.release_shared(np.array([1, 0, 1]), lens, table, free, count, shared, 4)
    assert free[:count].tolist() == [0, 5, 2] and shared.tolist() == [0] * 6 and lens.tolist() == [0, 9, 0]
    lens, free, count, shared = PO.release_shared(np.array([0, 1, 0]), lens, table, free, count, shared, 4)
    assert free[:count].tolist() == [0, 5, 2, 3, 4, 1]


def test_oracle_rotation_keeps_distances():
    rs = np.random.RandomState(1)
    q, k = rs.normal(size=(1, 1, 64)), rs.normal(size=(1, 1, 64))
    freq = [100.0 ** (-j / 16) for j in range(16)]
    for inter in (False, True):
        dots = [(PO.rotate(q, [p + 7], freq, inter)[0] * PO.rotate(k, [p], freq, inter)[0]).sum() for p in (0, 5, 1000)]
        assert np.ptp(dots) < 1e-10
        assert np.array_equal(PO.rotate(q, [0], freq, inter)[0], q)
    y = PO.rotate(q, [3], freq, weight=np.ones(64), eps=0.0)[0]
    assert abs((y * y).mean() - 1) < 1e-12
