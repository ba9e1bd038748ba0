"""Host-only checks of the paged cache's entry points and pins of its oracle."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from bit_quantized_kv_kvq_gb300.paged import PagedConfig, PagedLayout
from oracle import paged_oracle as PO


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kvq.lib()


GOOD = dict(num_layers=2, max_requests=8, num_kv_heads=4, head_dim=128, page_tokens=64, num_pages=100, max_pages=20,
            code=kvq.PAGE_INT8, dtype=1)


def config(**kw):
    return PagedConfig(**dict(GOOD, **kw))


def nbytes(lib, cfg):
    n = ctypes.c_size_t()
    return lib.kvq_paged_cache_bytes(ctypes.byref(cfg), ctypes.byref(n)), n.value


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_bytes_are_the_pages_scales_and_tails(lib, page, dim):
    st, n = nbytes(lib, config(page_tokens=page, head_dim=dim))
    tile = 2 * page * dim
    layer = 100 * 4 * tile + 100 * 4 * 2 * 4 + 8 * 4 * tile * 2
    assert st == 0 and 2 * layer <= n - 256 <= 2 * (layer + 3 * 256)


BAD = [(dict(num_layers=0), 1), (dict(max_requests=0), 1), (dict(max_requests=4097), 1), (dict(num_kv_heads=0), 1),
       (dict(head_dim=96), 2), (dict(page_tokens=48), 2), (dict(page_tokens=256), 2), (dict(num_pages=0), 1),
       (dict(num_pages=1 << 25), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 25), 1), (dict(max_pages=(1 << 25) - 1), 1), (dict(code=2), 1),
       (dict(dtype=0), 1), (dict(dtype=3), 1),
       (dict(max_requests=4096, max_pages=1 << 24), 2)]


@pytest.mark.parametrize("kw,status", BAD, ids=[str(b[0]) for b in BAD])
def test_bad_configs_are_rejected(lib, kw, status):
    assert nbytes(lib, config(**kw))[0] == status
    assert lib.kvq_last_error()


def test_create_rejects_bad_buffers_on_the_host(lib):
    cfg, h = config(), ctypes.c_void_p()
    assert lib.kvq_paged_cache_create(ctypes.byref(cfg), None, 1 << 30, None, ctypes.byref(h)) == 1
    assert lib.kvq_paged_cache_create(ctypes.byref(cfg), 0x1008, 1 << 30, None, ctypes.byref(h)) == 1
    assert lib.kvq_paged_cache_create(ctypes.byref(cfg), 0x10000, 100, None, ctypes.byref(h)) == 3
    assert lib.kvq_paged_cache_create(ctypes.byref(cfg), 0x10000, 1 << 30, None, None) == 1
    assert h.value is None


def test_null_handles_and_arrays_are_rejected(lib):
    z = [None] * 12
    assert lib.kvq_paged_reserve(None, 1, *z[:5], 1, *z[:6]) == 1
    assert lib.kvq_paged_release(None, 1, *z[:6]) == 1
    assert lib.kvq_paged_write(None, 0, 1, None, None, 512, 512, 1, None, None, None, None) == 1
    assert lib.kvq_paged_decode_attention(None, 0, 1, None, 512, 4, None, None, 1.0, None, 0, None, 0, None) == 1
    assert lib.kvq_paged_cache_status(None, None, None) == 1
    assert lib.kvq_paged_cache_destroy(None) == 0
    lo = PagedLayout()
    assert lib.kvq_paged_cache_get_layout(None, 0, ctypes.byref(lo)) == 1
    n = ctypes.c_size_t()
    assert lib.kvq_paged_decode_workspace_bytes(None, 4, ctypes.byref(n)) == 1


def prompt(lib, **kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, qs=1024, ks=256, vs=256, tokens=10, seqs=1, cu=0x40000, hq=8, hkv=2,
             d=128, dtype=1, scale=0.1, out=0x50000, status=None)
    a.update(kw)
    return lib.kvq_prompt_attention(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["tokens"], a["seqs"], a["cu"],
                                    a["hq"], a["hkv"], a["d"], a["dtype"], a["scale"], a["out"], a["status"], None)


PROMPT_BAD = [(dict(q=None), 1), (dict(k=0x20008), 1), (dict(qs=1020), 1), (dict(qs=1016), 1), (dict(ks=248), 1),
              (dict(tokens=-1), 1), (dict(seqs=0), 1), (dict(seqs=4097), 1), (dict(hq=7), 1), (dict(hkv=0), 1),
              (dict(d=96), 2), (dict(dtype=0), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(out=0x50004), 1),
              (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-0.1), 1),
              (dict(status=0x60002), 1), (dict(vs=1 << 40), 1)]


@pytest.mark.parametrize("kw,status", PROMPT_BAD, ids=[str(b[0]) for b in PROMPT_BAD])
def test_prompt_attention_refusals(lib, kw, status):
    before = kvq.kernel_launches()
    assert prompt(lib, **kw) == status
    assert kvq.kernel_launches() == before


def test_prompt_attention_of_no_tokens_does_nothing(lib):
    assert prompt(lib, tokens=0) == 0


# -- pins of the oracle ------------------------------------------------------
def test_e4m3_rounding_matches_torch():
    g = torch.Generator().manual_seed(1)
    y = torch.cat([torch.randn(20000, generator=g) * s for s in (1e-3, 0.02, 1.0, 100.0)]).clamp(-448, 448)
    mids = torch.tensor(PO.e4m3_values()[:127], dtype=torch.float32)
    y = torch.cat([y, (mids[1:] + mids[:-1]) / 2, -(mids[1:] + mids[:-1]) / 2, mids, -mids])
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(PO.to_e4m3(y.numpy()), want)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_page_grid_values_come_back_exactly(code):
    """Values on a page's own grid (largest magnitude Q) keep their codes."""
    rs = np.random.RandomState(3)
    vals = np.arange(-127, 128) if code == "int8" else PO.e4m3_values()[np.r_[0:127, 128:255]]
    x = vals[rs.randint(0, len(vals), (16, 64))].astype(np.float64)
    x[3, 5] = vals.max()
    for s in (1.0, 0.25, 2.0 ** -9):
        codes, scale = PO.quantize_page(x * s, code)
        assert scale == np.float32(s)
        assert np.array_equal(PO.page_values(codes, scale, code), x * s)


def test_page_scale_of_zeros_and_of_nonfinite_values():
    codes, s = PO.quantize_page(np.zeros((16, 64)), "int8")
    assert s == 0 and not codes.any()
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones((16, 64))
        x[2, 3] = bad
        for code in ("int8", "e4m3"):
            c, s = PO.quantize_page(x, code)
            assert np.isnan(PO.page_values(c, s, code)).all()


def test_oracle_attention_matches_torch_sdpa():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, 3, 20, 64, generator=g, dtype=torch.float64) for _ in range(3))
    want = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True)[0].transpose(0, 1).numpy()
    t = lambda x: x[0].transpose(0, 1).numpy()
    o, _, _ = PO.prompt_attention(t(q), t(k), t(v), [0, 20], 1 / 8.0)
    assert np.abs(o - want).max() < 1e-12


def test_oracle_reserve_and_release_by_hand():
    free = np.array([10, 11, 12, 13, 14], np.int32)
    table = np.full((2, 3), -1, np.int32)
    t, cu, slots, pos, lens, count = PO.reserve(np.array([3, 0]), np.array([2, 5]), np.array([[7, -1, -1], [-1] * 3]),
                                                free, 5, 8, 4)
    assert t.tolist() == [[7, 14, -1], [13, 12, -1]] and cu.tolist() == [0, 2, 7]
    assert slots.tolist() == [31, 56, 52, 53, 54, 55, 48, -1] and pos.tolist() == [3, 4, 0, 1, 2, 3, 4, -1]
    assert lens.tolist() == [5, 5] and count == 2
    lens, free, count = PO.release(np.array([0, 1]), lens, t, free, count, 4)
    assert lens.tolist() == [5, 0] and free[:count].tolist() == [10, 11, 13, 12]
    assert PO.reserve(np.array([3]), np.array([2]), table[:1], free, 0, 8, 4) is None
    assert PO.reserve(np.array([3]), np.array([2]), table[:1], free, 5, 1, 4) is None
