"""Where chunk attention's outputs may lie: anywhere but over the queries, between their rows included."""
import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from tests.test_gpu_paged import F16
from tests.test_gpu_paged_attend import Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 2, 37])
@pytest.mark.parametrize("gap", [0, 8, 40 * 256])
def test_out_beside_and_over_q(m, gap):
    f = Filled([50], [m], 4, 2, 64, 16, "int8", F16)
    row = 4 * 64
    want = f.attend()
    pool = torch.zeros(8 * 40 * (row + gap), dtype=F16, device="cuda")
    start = 3 * 40 * (row + gap)
    q = pool[start:].as_strided((m, 4, 64), (row + gap, 64, 1), start)
    q.copy_(f.q)
    kept = q.clone()
    size, last = m * row, start + (m - 1) * (row + gap) + row  # behind q's last element

    def at(offset):
        return pool[offset:offset + size].view(m, 4, 64)
    ends = [start - size, last] + ([start + row, start + row + gap - size] if gap >= size and m > 1 else [])
    for offset in ends:
        assert torch.equal(f.attend(q=q, out=at(offset)), want) and torch.equal(q, kept)
    for offset in (start, start - 8, start + 8, start - size + 8, last - 8, start + (m - 1) * (row + gap)):
        if any(start + i * (row + gap) < offset + size and offset < start + i * (row + gap) + row for i in range(m)):
            with pytest.raises(kvq.KVQError) as e:
                f.attend(q=q, out=at(offset))
            assert e.value.status == 1 and "overlap" in str(e.value)
    assert f.cache.status() == 0
