"""Sizes at the ends of what the entry points take."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
import oracle as O
from oracle import formats as F
from oracle import mxcast as M

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


@pytest.mark.parametrize("kind", ["mx", "w4a16", "w4a4"])
@pytest.mark.parametrize("tokens", [33, 128, 129])
@pytest.mark.parametrize("k", [512, 544])
def test_few_tokens_of_a_wide_output(kind, tokens, k):
    """Outputs enough to fill the card with large tiles, and tokens to fill
    a small one; sampled columns."""
    note(f"{kind} tokens={tokens} out=49300 k={k}")
    rng = np.random.default_rng(tokens)
    out = 49300
    at = np.unique(np.r_[0, 1, out - 140:out, rng.integers(0, out, 300)])
    unit, lo, hi = (32, 118, 134) if kind == "mx" else (16, 0, 127)
    def packed(rows):
        return rng.integers(0, 256, (rows, k // 2), dtype=np.uint8), rng.integers(lo, hi, (rows, k // unit), dtype=np.uint8)
    values = M.mxfp4_dequant if kind == "mx" else O.nvfp4_values
    w, x = packed(out), packed(tokens)
    wd, xd, one = [to_dev_u8(a) for a in w], [to_dev_u8(a) for a in x], to_dev_f32([1.0])
    xv = values(*x)
    if kind == "mx":
        y = nq.mxfp4_matmul(*xd, *wd)
    elif kind == "w4a4":
        y = nq.matmul_w4a4(*xd, one, *wd, one)
    else:
        bits = F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, k)))
        xv = F.bf16_bits_to_f64(bits)
        y = nq.matmul_w4a16(to_dev_bf16(bits), *wd, one)
    ref, mag = O.matmul(xv, values(w[0][at], w[1][at]))
    got = F.bf16_bits_to_f64(to_host_bits(y))[:, at]
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + (k + 3) * 2.0 ** -23 * mag * (1 + HALF))


# The most channels, altogether and in tiles.  All but some hundred activations
# (the last ones and the ends of what a pass of the waves takes among them) are
# zero, so that an fp32 sum has few terms.
K = 1 << 26


def _few_channels(rng, k):
    ends = [512 * 16, 512 * 12, 512 * 8, 512]
    at = np.r_[0:32, k - 64:k, [e - 1 for e in ends], ends, rng.integers(0, k // 32, 100) * 32 + rng.integers(0, 32, 100)]
    return np.unique(at)


@pytest.mark.parametrize("kind,tokens,out,K", [(kind, t, 20, K) for kind in ("mx", "w4a16", "w4a4") for t in (2, 20)] +
                         [(kind, 140, 150, (1 << 22) - cut) for kind in ("w4a16", "w4a4") for cut in (16, 64)] +
                         [("mx", 140, 150, (1 << 23) - cut) for cut in (32, 128)])
def test_product_of_the_most_channels(kind, tokens, out, K):
    note(f"{kind} tokens={tokens} out={out} k={K}")
    rng = np.random.default_rng(tokens)
    at = _few_channels(rng, K)
    where = torch.from_numpy(at).to(DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    unit = 32 if kind == "mx" else 16
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)
    lo, hi = (120, 135) if kind == "mx" else (1, 127)
    wp, wc = u8(0, 256, out, K // 2), u8(lo, hi, out, K // unit)

    def values(p, c):
        """float64 of the columns `at` of packed rows."""
        n = (host(p[:, where // 2]) >> (at % 2 * 4).astype(np.uint8)) & 15
        c = host(c[:, where // unit])
        scale = np.exp2(c.astype(np.float64) - 127) if kind == "mx" else F.E4M3_VALUES[c.astype(np.int64)]
        return F.e2m1_decode(n) * scale

    if kind == "w4a16":
        bits = F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, len(at))))
        x = torch.zeros((tokens, K), dtype=torch.bfloat16, device=DEV)
        x[:, where] = to_dev_bf16(bits)
        xv = F.bf16_bits_to_f64(bits)
        y = nq.matmul_w4a16(x, wp, wc, to_dev_f32([1.0]))
    else:
        xp, xc = torch.zeros((tokens, K // 2), dtype=torch.uint8, device=DEV), u8(lo, hi, tokens, K // unit)
        xp[:, where // 2] = u8(0, 256, tokens, len(at)) & torch.where(where % 2 == 0, 15, 240).to(torch.uint8)
        even = where[(where % 2 == 0) & torch.isin(where + 1, where)]        # bytes with both of their channels
        xp[:, even // 2] = u8(0, 256, tokens, len(even))
        xv = values(xp, xc)
        one = to_dev_f32([1.0])
        y = nq.mxfp4_matmul(xp, xc, wp, wc) if kind == "mx" else nq.matmul_w4a4(xp, xc, one, wp, wc, one)
    ref, mag = O.matmul(xv, values(wp, wc))
    got = F.bf16_bits_to_f64(to_host_bits(y))
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + (len(at) + 3) * 2.0 ** -23 * mag * (1 + HALF))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ld", [(1 << 22) - 8, 1 << 22])
def test_w4a16_of_rows_far_apart(ld):
    """Rows of x as far apart as 32-bit offsets within a tile reach, and farther."""
    note(f"w4a16 ldx={ld}")
    rng = np.random.default_rng(9)
    tokens, out, k = 260, 200, 80
    p, c = rng.integers(0, 256, (out, k // 2), dtype=np.uint8), rng.integers(0, 127, (out, k // 16), dtype=np.uint8)
    bits = F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, k)))
    x = torch.full((tokens, ld), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[:, :k] = to_dev_bf16(bits)
    y = nq.matmul_w4a16(x[:, :k], to_dev_u8(p), to_dev_u8(c), to_dev_f32([0.5]))
    ref, mag = O.matmul(F.bf16_bits_to_f64(bits), O.nvfp4_values(p, c, 0.5))
    got = F.bf16_bits_to_f64(to_host_bits(y))
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + (k + 3) * 2.0 ** -23 * mag * (1 + HALF))


@pytest.mark.parametrize("hidden,inter", [(K, 16), (16, K)])
def test_layer_of_the_most_channels(hidden, inter):
    """One side 2^26 channels, 16 on the other, two experts; in the second
    shape most rows of w1 are zero, so that few of h's values are not."""
    note(f"layer hidden={hidden} inter={inter}")
    rng = np.random.default_rng(7)
    tokens, experts = 2, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)
    at = _few_channels(rng, K)
    where = torch.from_numpy(at).to(DEV)
    p13, c13 = u8(0, 256, experts, 2, inter, hidden // 2), u8(48, 64, experts, 2, inter, hidden // 16)
    p2, c2 = u8(0, 256, experts, hidden, inter // 2), u8(48, 64, experts, hidden, inter // 16)
    s13, s2 = to_dev_f32([0.02, 0.03]), to_dev_f32([0.5, 0.25])
    x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=DEV)
    if hidden == K:
        x[:, where] = to_dev_bf16(F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, len(at)))))
        cols, rows, outs = where, torch.arange(inter, device=DEV), where
    else:
        x[:] = to_dev_bf16(F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, hidden))))
        keep = p13[:, 0, where].clone()
        p13[:, 0] = 0                                                # gate 0: silu 0
        p13[:, 0, where] = keep
        cols, rows, outs = torch.arange(hidden, device=DEV), where, torch.arange(hidden, device=DEV)
    ids = torch.tensor([[1], [0]], dtype=torch.int32, device=DEV)
    wt = to_dev_f32([[0.75], [1.5]])
    y = nq.moe_forward(x, ids, wt, p13, c13, s13, p2, c2, s2)

    def values(p, c, r, k):
        k = k.cpu().numpy()
        r = r.cpu().numpy()
        rt, kt = torch.from_numpy(r).to(DEV)[:, None], torch.from_numpy(k).to(DEV)[None]
        n = (host(p[rt, kt // 2]) >> (k % 2 * 4).astype(np.uint8)) & 15
        return F.e2m1_decode(n) * F.E4M3_VALUES[host(c[rt, kt // 16]).astype(np.int64)]

    u = 2.0 ** -23
    for t, e in ((0, 1), (1, 0)):
        xv = F.bf16_bits_to_f64(to_host_bits(x[t, cols]))
        w1, w3 = (values(p13[e, i], c13[e, i], rows, cols) * float(s13[e]) for i in (0, 1))
        w2 = values(p2[e], c2[e], outs, rows) * float(s2[e])
        gate, up = w1 @ xv, w3 @ xv
        n = len(xv) + 3
        eg, eu = n * u * (np.abs(w1) @ np.abs(xv)), n * u * (np.abs(w3) @ np.abs(xv))
        act = O.product.silu(gate)
        h = act * up
        eh = 1.1 * eg * (np.abs(up) + eu) + np.abs(act) * eu + 2.0 ** -20 * np.abs(h)
        ref = float(wt[t, 0]) * (w2 @ h)
        bound = float(wt[t, 0]) * (np.abs(w2) @ (eh + (2 * len(h) + 16) * u * np.abs(h)))
        got = F.bf16_bits_to_f64(to_host_bits(y[t, outs]))
        assert np.all(np.abs(got - ref) <= bound * (1 + HALF) + HALF * np.abs(ref))
    del p13, c13, p2, c2, x, y
    torch.cuda.empty_cache()
