"""Adapters at the ends of what the entry point takes."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq

import test_gpu_layer_lora as lora_test
from _gpu import DEV, need_gpu, note, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def test_adapters_of_more_tokens_than_a_launch_has_places():
    """The inner sums of 2^28 tokens, 32 a workgroup of 512 threads, would be 2^32
    threads.  The same 32768 tokens again and again, their adapters too: every
    repetition has the bits of the first, which is checked."""
    note("lora, 2^28 + 70 tokens")
    some, tokens, k, out, rank = 1 << 15, (1 << 28) + 70, 16, 8, 8
    c = lora_test.Case(1, some, out, k, 3, rank)
    times = -(-tokens // some)
    x = to_dev_bf16(c.x).repeat(times, 1)[:tokens]
    args = c.args()
    args[3] = args[3].repeat(times)[:tokens].contiguous()
    y = nq.matmul_w4a16_lora(x, *args)
    del x
    c.check(y[:some])
    for t in range(0, tokens, some):
        assert torch.equal(y[t:t + some], y[:min(some, tokens - t)]), t
    del y, args
    torch.cuda.empty_cache()
