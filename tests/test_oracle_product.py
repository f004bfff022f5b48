"""The MXFP4 quantizer, product and expert-layer oracle against independent
forms: rational brute force, torch's own softmax and matrix product, and
hand-made cases."""
from fractions import Fraction

import numpy as np
import torch

import oracle as O
from oracle import formats as F


def _bits(x):
    return F.f64_to_bf16_rne(np.asarray(x, dtype=np.float64))


def test_mxfp4_quantize_is_nearest_at_the_block_scale():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.laplace(0, 1, (20, 32)), rng.laplace(0, 1e-30, (4, 32)), rng.laplace(0, 1e30, (4, 32)),
                        np.ldexp(rng.integers(-64, 65, (8, 32)), -4)])
    bits = _bits(x)
    packed, code = O.mxfp4_quantize(bits)
    nib = F.unpack_nibbles(packed)
    v = F.bf16_bits_to_f64(bits)
    grid = [Fraction(float(m)) for m in F.E2M1_MAGNITUDES]
    for r in range(len(v)):
        amax = max(Fraction(abs(float(a))) for a in v[r])
        e = 0
        while Fraction(2) ** (e + 1) <= amax:
            e += 1
        while Fraction(2) ** e > amax:
            e -= 1
        assert int(code[r, 0]) == max(e - 2 + 127, 0)
        s = Fraction(2) ** (int(code[r, 0]) - 127)
        for a, n in zip(v[r], nib[r]):
            q = abs(Fraction(float(a))) / s
            d = [abs(q - g) for g in grid]
            best = min(d) if q <= 6 else d[7]
            near = [i for i in range(8) if d[i] == best]
            want = near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]
            assert int(n) & 7 == want and (int(n) >> 3) == int(np.signbit(a))


def test_mxfp4_quantize_edges():
    x = np.zeros((6, 32))
    x[1, 3] = np.inf
    x[2, 0] = np.nan
    x[3, 7] = 2.0 ** -133                  # the smallest bf16
    x[4, 9] = -F.bf16_bits_to_f64(np.uint16(0x7F7F))
    x[5, :2] = 7.0, -5.0                   # 7 saturates, 5 is a tie that goes to 4
    packed, code = O.mxfp4_quantize(_bits(x))
    assert code[:, 0].tolist() == [0, 255, 255, 0, 252, 127]
    assert not packed[:4].any()            # 2^-133 / 2^-127 is below a quarter
    assert F.unpack_nibbles(packed)[4, 9] == 0xF
    assert F.unpack_nibbles(packed)[5, :2].tolist() == [7, 0xE]


def test_round_trip_of_representable_blocks():
    rng = np.random.default_rng(4)
    p = rng.integers(0, 256, (9, 32), dtype=np.uint8)
    e = rng.integers(1, 250, (9, 2)).astype(np.uint8)
    p[:, 0] = 0x77                         # every block reaches its top binade
    p[:, 16] = 0x77
    from oracle.mxcast import mxfp4_dequant
    v = mxfp4_dequant(p, e)
    p2, e2 = O.mxfp4_quantize(_bits(v))
    assert np.array_equal(p, p2) and np.array_equal(e, e2)


def test_nvfp4_values_match_torch():
    rng = np.random.default_rng(5)
    p = rng.integers(0, 256, (3, 4, 24), dtype=np.uint8)
    c = rng.integers(0, 127, (3, 4, 3), dtype=np.uint8)
    s = rng.random(3)
    v = O.nvfp4_values(p, c, s)
    m = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    n = torch.from_numpy(np.stack([p & 15, p >> 4], -1).reshape(3, 4, 48).astype(np.int64))
    t = m[n & 7] * torch.where(n > 7, -1.0, 1.0)
    t = t * torch.from_numpy(c).view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    assert np.array_equal(v, (t * torch.from_numpy(s)[:, None, None]).numpy())


def test_route_against_torch_and_by_hand():
    rng = np.random.default_rng(6)
    z = rng.normal(0, 1, (40, 13))
    ids, w = O.moe_route(z, 4)
    v, i = torch.topk(torch.from_numpy(z), 4)
    assert np.array_equal(ids, i.numpy()) and np.allclose(w, torch.softmax(v, 1).numpy(), rtol=1e-14)
    _, wa = O.moe_route(z, 4, normalize=False)
    assert np.allclose(wa, torch.softmax(torch.from_numpy(z), 1).gather(1, i).numpy(), rtol=1e-13)
    n, inf = np.nan, np.inf
    ids, w = O.moe_route(np.array([[1, 1, 0, 1], [n, -inf, 2, n], [-inf, n, n, -inf], [inf, 0, inf, n]]), 3)
    assert ids.tolist() == [[0, 1, 3], [2, -1, -1], [-1, -1, -1], [0, 2, 1]]
    assert np.allclose(w[0], 1 / 3) and w[1].tolist() == [1, 0, 0] and not w[2].any()
    assert w[3].tolist() == [0.5, 0.5, 0]


def test_moe_forward_against_torch():
    rng = np.random.default_rng(7)
    x = rng.normal(0, 1, (5, 8))
    w13, w2 = rng.normal(0, 1, (3, 2, 6, 8)), rng.normal(0, 1, (3, 8, 6))
    ids = np.array([[0, 1], [2, 2], [-1, 0], [3, 7], [1, 0]])
    wt = rng.random((5, 2))
    y, mag = O.moe_forward(x, ids, wt, w13, w2)
    X, A, B = (torch.from_numpy(a) for a in (x, w13, w2))
    every = torch.nn.functional.silu(torch.einsum("eid,td->tei", A[:, 0], X)) * torch.einsum("eid,td->tei", A[:, 1], X)
    every = torch.einsum("edi,tei->ted", B, every)
    ref = torch.zeros(5, 8, dtype=torch.float64)
    for t in range(5):
        for s in range(2):
            if 0 <= ids[t, s] < 3:
                ref[t] += wt[t, s] * every[t, ids[t, s]]
    assert np.allclose(y, ref.numpy(), rtol=1e-12, atol=1e-12) and not y[3].any()
    assert np.all(mag >= np.abs(y) - 1e-12)
