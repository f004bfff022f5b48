"""What the expert layer hands from its first product to the second,
h = weight * scale_2 * silu(gate) * up, is a float32 value: inputs whose exact
results show every one of its 24 bits, and values at the end of its range."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
from oracle import formats as F

from _gpu import DEV, need_gpu, note, to_dev_bf16, to_dev_f32, to_dev_u8, to_host_bits

pytestmark = pytest.mark.gpu

ONE, MINUS, HALF, SIX = 2, 10, 1, 7          # E2M1 nibbles of 1, -1, 0.5 and 6
CODE_ONE = 0x38                              # E4M3 1.0


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _bits(x):
    return F.f64_to_bf16_rne(np.asarray(x, dtype=np.float64))


class Layer:
    """Experts of E2M1 values alone: every block and tensor scale is 1."""

    def __init__(self, tokens, hidden, inter, experts):
        self.x = np.zeros((tokens, hidden))
        self.w13 = np.zeros((experts, 2, inter, hidden), np.uint8)
        self.w2 = np.zeros((experts, hidden, inter), np.uint8)
        self.weights = np.ones((tokens, 1), np.float32)

    def run(self, ids):
        def packed(n):
            return to_dev_u8(F.pack_nibbles(n)), to_dev_u8(np.full(n.shape[:-1] + (n.shape[-1] // 16,), CODE_ONE, np.uint8))
        ones = to_dev_f32(np.ones(len(self.w2)))
        y = nq.moe_forward(to_dev_bf16(_bits(self.x)), torch.from_numpy(ids.astype(np.int32)[:, None]).to(DEV),
                           to_dev_f32(self.weights), *packed(self.w13), ones, *packed(self.w2), ones)
        return to_host_bits(y)


@pytest.mark.parametrize("hidden,inter", [(64, 16), (96, 48), (64, 544), (80, 2048)])
@pytest.mark.parametrize("tokens,experts", [(1, 1), (5, 1), (9, 2), (64, 3)])
def test_every_bit_of_a_float32_counts(tokens, experts, hidden, inter):
    """gate = 64, so that silu(gate) is 64 (1 + exp(-64) is 1 in float32); up
    = 1 + r 2^-15 + j 2^-23, r a token's own 8 bits, j a channel's, so that all
    24 bits are in use; an output is the difference of two channels, 64 (j_a -
    j_b) 2^-23.  Every product, sum and difference on the way is a multiple of
    2^-17 below 2^7 (of 2^-23 below 2 before silu), which float32 holds exactly
    in any order, and the result has 8 bits: it must be met exactly.  tokens
    and their weights differ by powers of two as well."""
    note(f"layer bits tokens={tokens} hidden={hidden} inter={inter} experts={experts}")
    rng = np.random.default_rng(tokens + inter)
    L = Layer(tokens, hidden, inter, experts)
    j = rng.integers(0, 256, (experts, inter))
    two = 2.0 ** rng.integers(-3, 4, tokens)
    L.x[:, 0] = two                                                  # up's leading 1
    for b in range(8):
        L.x[:, 1 + b] = two * 2.0 ** (b - 23)
        L.w13[:, 1, :, 1 + b] = np.where(j >> b & 1, ONE, 0)
    L.x[:, 9] = two * 2.0 ** -15 * rng.integers(128, 256, tokens)
    L.w13[:, 1, :, [0, 9]] = ONE
    L.x[:, 10] = 64.0
    L.w13[:, 0, :, 10] = ONE
    L.weights[:, 0] = 2.0 ** rng.integers(-3, 4, tokens)
    at = np.stack([rng.permutation(inter)[:2] for _ in range(experts * hidden)]).reshape(experts, hidden, 2)
    e, o = np.arange(experts)[:, None], np.arange(hidden)[None]
    L.w2[e, o, at[..., 0]] = ONE
    L.w2[e, o, at[..., 1]] = MINUS
    ids = rng.integers(0, experts, tokens)
    diff = j[e, at[..., 0]] - j[e, at[..., 1]]                       # [experts, hidden]
    want = diff[ids] * 2.0 ** -17 * (two * L.weights[:, 0])[:, None]
    got = F.bf16_bits_to_f64(L.run(ids))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("tokens", [1, 6])
def test_largest_floats_and_infinity(tokens):
    """h above the largest bf16 but a float32 stays one, and an h that
    overflows is infinite, not NaN; neither reaches another token."""
    note(f"layer range tokens={tokens}")
    L = Layer(tokens, 32, 16, 1)
    L.w13[0, 0, 5, 0] = ONE                                          # gate and up of channel 5; the others are zero
    L.w13[0, 1, 5, 1:3] = ONE
    L.w2[0, :, 5] = np.resize([HALF, ONE, SIX, MINUS], 32)
    L.x[:, :3] = 2.0, 3.0, 0.25
    L.x[0, :3] = 2.0 ** 64, 2.0 ** 64, -2.0 ** 53                    # h = (2 - 2^-10) 2^127: bf16's largest is (2 - 2^-7) 2^127
    ids = np.zeros(tokens)
    w2 = np.resize([0.5, 1.0, 6.0, -1.0], 32)
    got = F.bf16_bits_to_f64(L.run(ids))
    # 0.5 h rounds to 2^127; h, -h and 6 h are above the largest bf16
    assert np.array_equal(got[0], np.where(w2 == 0.5, 2.0 ** 127, np.sign(w2) * np.inf))
    small = 2.0 / (1.0 + np.exp(-2.0)) * 3.25
    assert np.all(np.abs(got[1:] - w2 * small) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(w2 * small))
    L.x[0, :3] = 2.0 ** 64, 2.0 ** 64, 0.0                           # h = 2^128
    got = F.bf16_bits_to_f64(L.run(ids))
    assert np.array_equal(got[0], np.sign(w2) * np.inf)
    assert np.all(np.abs(got[1:] - w2 * small) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(w2 * small))
