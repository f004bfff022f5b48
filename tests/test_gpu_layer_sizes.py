"""The expert layer over sorted tokens and the adapters at the ends of what they
take, and on both sides of each size at which their kernels change."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq

import test_gpu_layer_experts as experts_test
import test_gpu_layer_lora as lora_test
from _gpu import DEV, need_gpu, note, to_dev_bf16, to_dev_f32, to_dev_u8

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


@pytest.mark.parametrize("tokens", [3, 17, 40])
@pytest.mark.parametrize("k", [1024, 528])
def test_adapters_of_tokens_far_apart(tokens, k):
    """x's rows are 8 MiB apart, too far for tiles: any number of tokens goes through
    the streaming kernels, 4, 8 or 16 at a time (k off 32: 4 or 16)."""
    note(f"lora, {tokens} tokens far apart, k={k}")
    c = lora_test.Case(tokens, tokens, 150, k, 5, 40)
    x = torch.full((tokens, 1 << 22), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[:, :k] = to_dev_bf16(c.x)
    c.check(c.run(x=x[:, :k]))


# rows an expert at the ends of the tiles' forms (32, 64, 96, 128) and of a band (256)
COUNTS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159, 160, 161, 255, 256, 257, 511, 512, 513]


@pytest.mark.parametrize("hidden,inter", [(64, 64), (80, 48), (272, 144)])
def test_rows_of_an_expert(hidden, inter):
    note(f"layer, counts of rows, {hidden} -> {inter}")
    of = np.repeat(np.arange(len(COUNTS)), COUNTS)
    c = experts_test.Case(hidden, len(of), hidden, inter, len(COUNTS), 1,
                          lambda r: r.permutation(of)[:, None])
    c.check(c.run())


@pytest.mark.parametrize("more", [1, 2, 70, 8192])
def test_results_do_not_depend_on_the_pass(more):
    """8192 tokens of 16 places are a pass; those of the second repeat the first's."""
    note(f"layer, second pass of {more} tokens")
    first = 8192
    c = experts_test.Case(3, first + more, 48, 32, 8, 16)
    for a in (c.x, c.ids, c.wt):
        a[first:] = a[:more]
    y = c.run()
    assert torch.equal(y[first:], y[:more])
    c.check(y)


@pytest.mark.parametrize("hidden,inter", [(1 << 17, 16), (16, 1 << 17), ((1 << 17) - 16, 48), (48, (1 << 17) - 48)])
def test_the_longest_sides(hidden, inter):
    note(f"layer, {hidden} -> {inter}")
    c = experts_test.Case(1, 70, hidden, inter, 2, 1)
    c.check(c.run())


def test_weights_past_four_gigabytes():
    """1024 experts: the last ones' packed weights begin 8.6 and 4.3 GB on, of which
    hidden is off the stages' 64, so that scales are copied as well."""
    note("layer, weights past 4 GiB")
    tokens, hidden, inter, experts = 100, 8208, 1024, 1024
    some = np.array([0, 511, experts - 2, experts - 1])
    c = experts_test.Case(7, tokens, hidden, inter, len(some), 3)
    dev = []
    for a in c.w:
        whole = torch.zeros((experts, *a.shape[1:]), dtype=torch.float32 if a.dtype == np.float32 else torch.uint8, device=DEV)
        whole[torch.from_numpy(some).to(DEV)] = to_dev_f32(a) if a.dtype == np.float32 else to_dev_u8(a)
        dev.append(whole)
    assert dev[3][-1].data_ptr() - dev[3].data_ptr() > 1 << 32
    ids = np.where(c.ids < 0, -1, some[c.ids]).astype(np.int32)
    y = nq.moe_forward_sorted(to_dev_bf16(c.x), torch.from_numpy(ids).to(DEV), to_dev_f32(c.wt), *dev)
    c.check(y)
    del dev
    torch.cuda.empty_cache()
