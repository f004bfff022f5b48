"""How many bits the expert layer over sorted tokens keeps between its products.

silu * up and an expert's row are rounded to fp16, 2^-11 of their value at most, y to
bf16, 2^-8 of its own; sums of n products in fp32 are off by n 2^-23 of the sum of
magnitudes.  A silu * up 2^28 and more below the largest of its row is off by 2^-38
of that one: half of fp16's last step where the largest is 2^14 or more, 2^-39, when it
is stored, and again when the row is brought to one power of two."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import formats as F
from oracle import layer as L
from oracle.product import silu

import test_gpu_layer_experts as experts_test
from _gpu import need_gpu, note, to_dev_f32, to_dev_u8, to_host_bits

pytestmark = pytest.mark.gpu

HALF, EPS, FP16 = 2.0 ** -8, 2.0 ** -23, 2.0 ** -11


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _case(tokens, hidden, inter, experts, top_k, seed):
    c = experts_test.Case(seed, tokens, hidden, inter, experts, top_k)
    c.ids[c.ids < 0] = 0
    return c


def _want(c):
    """(y, bound before y's rounding)"""
    p13, c13, s13, p2, c2, s2 = c.w
    x, wt = F.bf16_bits_to_f64(c.x), c.wt.astype(np.float64)
    w13, w2 = O.nvfp4_values(p13, c13, s13), O.nvfp4_values(p2, c2, s2)[:, 0]
    with np.errstate(over="ignore"):
        ref, off = L.moe_forward_sorted(x, c.ids, wt, w13, w2, EPS, FP16 + 32 * EPS, FP16)
        for e in range(c.experts):
            t, s = np.nonzero(c.ids == e)
            if t.size:
                top = np.abs(silu(x[t] @ w13[e, 0].T) * (x[t] @ w13[e, 1].T)).max(1) * 1.01
                np.add.at(off, t, (wt[t, s] * top * 2.0 ** -38)[:, None] * np.abs(w2[e]).sum(1))
    return ref, off


def _check(c):
    got = F.bf16_bits_to_f64(to_host_bits(c.run()))
    ref, off = _want(c)
    bound = HALF * np.abs(ref) + off * (1 + HALF) + 2.0 ** -120
    assert np.all(np.abs(got - ref) <= bound), f"{np.max(np.abs(got - ref) / bound):.3f} of the bound"
    return got, ref


# rows an expert up to 32, 64, 96, 128 and beyond; inter off 32 and 64
SIZES = [(70, 64, 48, 8), (100, 96, 64, 2), (180, 48, 16, 2), (120, 64, 176, 1), (700, 128, 80, 3)]


@pytest.mark.parametrize("tokens,hidden,inter,experts", SIZES)
@pytest.mark.parametrize("spread", [0, 12])
def test_an_output_of_one_channel(tokens, hidden, inter, experts, spread):
    """W2's row o is 1 in channel o mod inter alone, so that y is weight * silu * up of
    that channel and each rounding shows by itself; the channels' sizes differ by up
    to 2^(2 spread)."""
    note(f"layer, one channel an output, {tokens} tokens, {hidden} -> {inter}, spread {spread}")
    c = _case(tokens, hidden, inter, experts, 1, tokens)
    rng = np.random.default_rng(tokens)
    c.wt = (0.5 + rng.random((tokens, 1))).astype(np.float32)
    if spread:                                                       # scales of gate and up rows, 2^-spread .. 1
        c.w[1][:] = (0x38 - 8 * (rng.integers(0, spread + 1, (experts, 2, inter, 1)) // 2)).astype(np.uint8)
    nibbles = np.zeros((experts, hidden, inter), np.uint8)
    nibbles[:, np.arange(hidden), np.arange(hidden) % inter] = 2     # E2M1 1.0
    c.w[3] = F.pack_nibbles(nibbles)[:, None]
    c.w[4] = np.full((experts, 1, hidden, inter // 16), 0x38, np.uint8)
    c.w[5] = np.ones(experts, np.float32)
    c.dev = [to_dev_f32(a) if a.dtype == np.float32 else to_dev_u8(a) for a in c.w]
    _check(c)


@pytest.mark.parametrize("tokens,experts,top_k", [(100, 4, 1), (300, 8, 4), (1000, 4, 2)])
def test_error_over_many_outputs(tokens, experts, top_k):
    """Rounding errors are spread over half a step and independent: over many outputs
    y's own makes 2^-8 / sqrt(3) of y at most, and each of the two others an eighth of
    that of what it rounds, whose squares' sum over channels or places is not above the
    outputs' (signs are as likely either way)."""
    note(f"layer, error of many outputs, {tokens} tokens")
    c = _case(tokens, 512, 256, experts, top_k, tokens + 1)
    got, ref = _check(c)
    assert np.linalg.norm(got - ref) <= np.sqrt((1 + 2 * 2.0 ** -6) / 3) * HALF * np.linalg.norm(ref)


def test_infinities_beside_small_values():
    """A channel that overflows is infinite, in a row where others are 2^-200 of the
    largest finite one: it stays infinite (or NaN, with its sign lost), in its token."""
    note("layer, infinities beside small values")
    c = _case(80, 64, 96, 2, 1, 5)
    clean = c.run()
    c.x[3, :] = 0x7F00                                               # 1.7e38, all
    y = c.run()
    same = [t for t in range(80) if t != 3]
    assert torch.equal(y[same], clean[same]) and not torch.isfinite(y[3]).all()
