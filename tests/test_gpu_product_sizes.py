"""Sizes at the ends of what the entry points take."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
import oracle as O
from oracle import formats as F

from _gpu import DEV, need_gpu, note, host, to_dev_bf16, to_dev_f32, to_dev_u8, to_host_bits

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8           # half a bf16 step, relative


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("out", [(1 << 31) - 16, (1 << 31) - 256])
def test_product_of_the_most_outputs(out):
    """17 tokens, 16 channels, 2^31 columns a row of y: by the streaming
    kernels, and in tiles, whose last one ends with the 32-bit range.  Columns
    past the last output stay as they were."""
    tokens, k, ld = 17, 16, 1 << 31
    note(f"w4a16 tokens={tokens} out={out}")
    rng = np.random.default_rng(3)
    at = np.unique(np.r_[0:40, out // 2:out // 2 + 40, out - 600:out, rng.integers(0, out, 500)])
    where = torch.from_numpy(at).to(DEV)
    p, c = (rng.integers(0, 256, (len(at), 8), dtype=np.uint8), rng.integers(0, 127, (len(at), 1), dtype=np.uint8))
    wp = torch.zeros((out, 8), dtype=torch.uint8, device=DEV)
    wc = torch.zeros((out, 1), dtype=torch.uint8, device=DEV)
    wp[where], wc[where] = to_dev_u8(p), to_dev_u8(c)
    bits = F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, k)))
    y = torch.full((tokens, ld), 7.0, dtype=torch.bfloat16, device=DEV)
    nq.matmul_w4a16(to_dev_bf16(bits), wp, wc, to_dev_f32([0.5]), out=y[:, :out])
    ref, mag = O.matmul(F.bf16_bits_to_f64(bits), O.nvfp4_values(p, c, 0.5))
    for t in range(tokens):
        row = y[t]
        got = F.bf16_bits_to_f64(to_host_bits(row[where]))
        assert np.all(np.abs(got - ref[t]) <= HALF * np.abs(ref[t]) + (k + 3) * 2.0 ** -23 * mag[t] * (1 + HALF))
        assert bool((row[out:] == 7).all())
        row[where] = 0
        assert not bool(row[:out].any())
    del y, wp, wc
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens,experts,top_k", [((1 << 26) + 5, 2, 1), ((1 << 26) - 3, 1, 1)])
def test_route_of_more_tokens_than_a_launch_has_places(tokens, experts, top_k):
    """A wave a token would be 2^32 threads and more."""
    note(f"route tokens={tokens}")
    z = torch.zeros((tokens, experts), dtype=torch.float32, device=DEV)
    rng = np.random.default_rng(tokens)
    at = np.r_[0, 1, tokens - 2, tokens - 1, rng.choice(tokens, 2000, replace=False)]
    some = rng.normal(0, 1, (len(at), experts)).astype(np.float32)
    where = torch.from_numpy(at).to(DEV)
    z[where] = torch.from_numpy(some).to(DEV)
    ids, w = nq.moe_route(z, top_k)
    ri, rw = O.moe_route(host(z[where]), top_k, True)
    assert np.array_equal(host(ids[where]), ri) and np.array_equal(host(w[where]), rw.astype(np.float32))
    assert int(ids.min()) == 0 and int(ids.max()) < experts and bool((w == 1).all())
