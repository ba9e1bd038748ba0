"""The prompt attention's bounded waits against its longest block. The longest
prompt would take minutes, so its block is reckoned from a shorter one's tiles."""
import math
import os
import re

import pytest
import torch

import bit_quantized_kv_kvq_gb300 as kvq
from bit_quantized_kv_kvq_gb300 import workloads as W
from tests import kvq_check as K
from tests.test_gpu_prompt_attention import BF16, ints

pytestmark = pytest.mark.gpu
CSRC = os.path.join(os.path.dirname(kvq.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def milliseconds(call):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


def test_the_waits_outlast_the_longest_block():
    polls = 1 << int(re.search(r"kWaitLimit = 1 << (\d+);", source("common.cuh")).group(1))
    polls *= int((re.search(r"kPolls = (\d+) \* kWaitLimit;", source("prompt_attn.cu")) or [None, 1])[1])
    longest = 1 << int(re.search(r"max_tokens > 1 << (\d+)", source("kvq_paged.cu")).group(1))
    # what a poll takes, by a wait that runs out (a few milliseconds)
    cache = K.make_gpu_cache(W.TINY_Q8, 300)
    cache.selftest_wait_timeout(100)
    poll = milliseconds(lambda: cache.selftest_wait_timeout(2000)) / 2000
    with pytest.raises(kvq.KVQError):
        cache.status()
    # a pair of units' key tiles: 128 query rows of two heads, 128 keys each
    t = 1 << 19
    x = torch.randn(t, 4, 128, device="cuda", dtype=BF16)
    cu = ints([0, t])
    def run():
        kvq.prompt_attention(x[:, :2], x[:, 2:3], x[:, 3:], cu, 1 / math.sqrt(128))
    run()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = t // 128
    tile = milliseconds(run) * sms / (rows * (rows + 1) / 2)
    # twice the block at the clocks of now: clocks fall under the power limit
    assert polls * poll > 2 * tile * (longest // 128), (poll, tile)
