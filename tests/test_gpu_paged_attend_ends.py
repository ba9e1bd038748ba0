"""Chunk attention in a bf16 cache: a tile that the request's end or a page out of range leaves
partly empty has no open rows, and its weights are fp16."""
import pytest
import torch

from tests.test_gpu_paged import BF16
from tests.test_gpu_paged_attend import Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code,d", [("int8", 128), ("e4m3", 64), ("int8", 64), ("e4m3", 128)])
@pytest.mark.parametrize("page,lens", [(16, [16, 48, 144, 400]), (64, [64, 192, 320, 1088]), (32, [96, 32, 1120, 224])])
def test_weights_of_11_bits_up_to_the_end(code, d, page, lens):
    new = [min(n, m) for n, m in zip(lens, (16, 40, 7, 64))]
    f = Filled(lens, new, 8, 2, d, page, code, BF16, seed=page)
    f.check(f.attend(), weight=2.0 ** -11)
    assert f.cache.status() == 0


@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_weights_of_11_bits_beside_a_page_out_of_range(bad):
    """The pages before it, as the only ones that the rows see."""
    f = Filled([128], [100], 8, 2, 64, 16, "int8", BF16, seed=3)
    want = f.attend()
    f.table[0, 7] = bad
    out = f.attend()
    assert torch.equal(out[:112 - 28], want[:112 - 28])  # tokens at positions below 112
    with pytest.raises(Exception):
        f.cache.status()
