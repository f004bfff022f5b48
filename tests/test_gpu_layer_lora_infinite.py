"""An infinite value of an adapter's B: u times it is infinite, with the product's
sign, wherever u is not zero, for any number of tokens.  Whole numbers, so that all
else is exact."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq

from _gpu import DEV, need_gpu, note

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# streamed; small tiles, whole and with the channels split; large tiles
@pytest.mark.parametrize("tokens,k,out,rank", [(3, 64, 80, 8), (16, 64, 80, 40), (48, 64, 80, 40), (40, 4096, 96, 72),
                                               (300, 144, 80, 24), (4096, 64, 4096, 16)])
@pytest.mark.parametrize("one", [False, True])
def test_infinite_b(tokens, k, out, rank, one):
    """one: all tokens of one adapter."""
    note(f"lora, infinite B, {tokens} tokens, {k} -> {out}, rank {rank}, one adapter {one}")
    n = 3
    rng = np.random.default_rng(tokens + rank)
    x, a = np.zeros((tokens, k)), np.zeros((n, rank, k))
    at = rng.integers(0, k, (tokens, 2))                             # two channels a token, of two ranks or one
    x[np.arange(tokens), at[:, 0]] = rng.integers(1, 9, tokens)
    x[np.arange(tokens), at[:, 1]] = -rng.integers(1, 9, tokens)
    a[:, np.arange(k) % rank, np.arange(k)] = 1
    b = rng.integers(-9, 10, (n, out, rank)).astype(np.float64)
    b[1, 5::16, at[0, 0] % rank] = np.inf
    b[1, 7::16, at[1, 1] % rank] = -np.inf
    ids = np.full(tokens, 1) if one else rng.integers(-1, n, tokens)
    ids[:2] = 1
    dev = lambda v, d: torch.from_numpy(v).to(DEV, d)
    y = nq.matmul_w4a16_lora(dev(x, torch.bfloat16), torch.zeros(out, k // 2, dtype=torch.uint8, device=DEV),
                             torch.zeros(out, k // 16, dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV),
                             dev(ids, torch.int32), dev(a, torch.bfloat16), dev(b, torch.bfloat16),
                             torch.full((n,), 2.0, device=DEV)).float().cpu().numpy()
    want = np.zeros((tokens, out))
    for j in range(n):
        t = np.flatnonzero(ids == j)
        u = 2 * (x[t] @ a[j].T)
        with np.errstate(invalid="ignore"):                          # (0 times infinity)
            for r in range(rank):
                want[t] += u[:, r, None] * b[j, :, r]
    assert np.isinf(want[:2]).any()
    assert np.array_equal(y, want, equal_nan=True), f"{(~((y == want) | (np.isnan(y) & np.isnan(want)))).sum()} outputs differ"
