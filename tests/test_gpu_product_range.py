"""The whole range of the packed products' and the expert layer's operands:
block scales of every exponent and opposite extremes, activations that are
infinite, NaN, subnormal or large, NaN among the router's weights, and layers
of the sizes that expert sets have, against float64.

Bounds are those of test_gpu_product: k 2^-23 of the sum of magnitudes for the
fp32 sums (3 more for tensor scales and partial tiles) and half a bf16 step,
2^-8 of the value, for the result."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
import oracle as O
from oracle import formats as F
from oracle import mxcast as M

from _gpu import DEV, need_gpu, note, to_dev_bf16, to_dev_f32, to_dev_u8, to_host_bits

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8           # half a bf16 step, relative


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _values(y):
    return F.bf16_bits_to_f64(to_host_bits(y))


def _near(got, x, w, scale=1.0, tiny=0.0):
    ref, mag = O.matmul(x, w * scale)
    bound = HALF * np.abs(ref) + (x.shape[1] + 3) * 2.0 ** -23 * mag * (1 + HALF) + tiny
    assert np.all(np.abs(got - ref) <= bound), f"max excess {np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3f}"


# ------------------------------------------------------------- MXFP4 ----
# tokens and k: both streaming forms, small tiles with rows of scales as they
# are and copied, large tiles
MX = [(1, 512), (16, 544), (20, 4096), (32, 4640), (33, 1024), (200, 544), (130, 4096)]


def _codes(rng, tokens, out, blocks, total):
    """E8M0 codes of both sides over the whole range, opposite in every block:
    their sum is `total` plus up to 3 either way."""
    a = rng.integers(0, 255, blocks)
    a[:2] = 0, 254
    def side(rows, centre):
        return np.clip(centre + rng.integers(-1, 2, (rows, blocks)), 0, 254).astype(np.uint8)
    return side(tokens, a[None]), side(out, np.clip(total - a, 0, 254)[None])


@pytest.mark.parametrize("tokens,k", MX)
def test_mx_scales_of_opposite_extremes(tokens, k):
    note(f"mx opposite scales tokens={tokens} k={k}")
    rng = np.random.default_rng(tokens + k)
    out = 150
    xp, wp = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (tokens, out))
    xe, we = _codes(rng, tokens, out, k // 32, 254)
    y = nq.mxfp4_matmul(*[to_dev_u8(a) for a in (xp, xe, wp, we)])
    _near(_values(y), M.mxfp4_dequant(xp, xe), M.mxfp4_dequant(wp, we))


@pytest.mark.parametrize("tokens,k", MX)
@pytest.mark.parametrize("total", [140, 370])
def test_mx_scales_of_small_and_large_products(tokens, k, total):
    """Sums near 2^-114 and 2^116 times k, made of scales from end to end."""
    note(f"mx scales total={total} tokens={tokens} k={k}")
    rng = np.random.default_rng(tokens + k + total)
    out = 70
    xp, wp = (rng.integers(0, 256, (r, k // 2), dtype=np.uint8) for r in (tokens, out))
    a = rng.integers(max(0, total - 254), min(254, total) + 1, k // 32)
    xe, we = (np.repeat(c.astype(np.uint8)[None], r, 0) for c, r in ((a, tokens), (total - a, out)))
    if total > 254:                                                  # sums stay below 2^128
        xp, wp = xp & 0x9B, wp & 0x9B                                # |e2m1| up to 1.5
        xp[:, 64:], wp[:, 64:] = 0, 0
    y = nq.mxfp4_matmul(*[to_dev_u8(v) for v in (xp, xe, wp, we)])
    assert bool(torch.isfinite(y).all())
    _near(_values(y), M.mxfp4_dequant(xp, xe), M.mxfp4_dequant(wp, we))


@pytest.mark.parametrize("tokens", [2, 40])
def test_mx_overflow_is_infinite_and_underflow_zero(tokens):
    note(f"mx overflow tokens={tokens}")
    k, out = 128, 64
    xp, wp = np.zeros((tokens, k // 2), np.uint8), np.zeros((out, k // 2), np.uint8)
    xp[:, 20], wp[:, 20] = 0x02, 0x02                                # one product of 1 x 1
    wp[1::2, 20] = 0x0A
    xe, we = np.full((tokens, 4), 254, np.uint8), np.full((out, 4), 254, np.uint8)
    args = [to_dev_u8(v) for v in (xp, xe, wp, we)]
    sign = np.resize([1.0, -1.0], out)[None]
    assert np.array_equal(_values(nq.mxfp4_matmul(*args)), np.repeat(sign * np.inf, tokens, 0))
    for e in (args[1], args[3]):
        e.zero_()
    assert not _values(nq.mxfp4_matmul(*args)).any()


# ------------------------------------------------- bf16 activations ----
# tokens, k: 4, 8 and 16 tokens a workgroup, k off 32, both tile sizes' paths
A16 = [(1, 512), (6, 544), (16, 1024), (3, 528), (13, 528), (17, 512), (70, 528), (300, 1024)]


def _weight(rng, out, k, lo=0, hi=127):
    p = rng.integers(0, 256, (out, k // 2), dtype=np.uint8)
    return p, rng.integers(lo, hi, (out, k // 16), dtype=np.uint8)


def _acts(rng, tokens, k):
    return F.f64_to_bf16_rne(rng.normal(0, 1, (tokens, k)))


@pytest.mark.parametrize("tokens,k", A16)
def test_w4a16_subnormal_and_mixed_activations(tokens, k):
    """Subnormal bf16 activations count with their exact values; alone and
    among others of every exponent whose products fp32 holds."""
    note(f"w4a16 subnormal tokens={tokens} k={k}")
    rng = np.random.default_rng(tokens + k)
    out = 100
    p, c = _weight(rng, out, k, 0x70)                                # v up to 2688, blocks of 128 and more
    s2 = 2.0 ** 60
    w = O.nvfp4_values(p, c)
    args = [to_dev_u8(p), to_dev_u8(c), to_dev_f32([s2])]
    sub = rng.integers(0, 0x80, (tokens, k)).astype(np.uint16) | (rng.integers(0, 2, (tokens, k)) << 15).astype(np.uint16)
    _near(_values(nq.matmul_w4a16(to_dev_bf16(sub), *args)), F.bf16_bits_to_f64(sub), w, s2)
    mixed = sub.copy()
    for t in range(0, tokens, 2):                                    # each such row about one exponent
        e = int(rng.integers(1, 100))
        mixed[t] = (rng.integers(0, 0x80, k) | (e + rng.integers(0, 2, k)) << 7 | rng.integers(0, 2, k) << 15).astype(np.uint16)
    _near(_values(nq.matmul_w4a16(to_dev_bf16(mixed), *args)), F.bf16_bits_to_f64(mixed), w, s2)


@pytest.mark.parametrize("tokens,k", A16)
def test_w4a16_infinities_and_nan_stay_in_their_row(tokens, k):
    note(f"w4a16 inf and nan tokens={tokens} k={k}")
    rng = np.random.default_rng(tokens * 3 + k)
    out = 100
    p, c = _weight(rng, out, k, 1)
    w = O.nvfp4_values(p, c)
    args = [to_dev_u8(p), to_dev_u8(c), to_dev_f32([0.01])]
    bits = _acts(rng, tokens, k)
    plain = nq.matmul_w4a16(to_dev_bf16(bits), *args)
    for pattern in (0x7FC0, 0x7F81, 0x7F80, 0xFF80):
        for row, ch in ((0, 0), (tokens // 2, k - 1), (tokens - 1, k // 2)):
            b = bits.copy()
            b[row, ch] = pattern
            y = nq.matmul_w4a16(to_dev_bf16(b), *args)
            got = _values(y)[row]
            if pattern in (0x7FC0, 0x7F81):
                assert np.isnan(got).all()
            else:
                with np.errstate(invalid="ignore"):
                    want = F.bf16_bits_to_f64(np.uint16(pattern)) * w[:, ch]
                assert np.array_equal(got, want, equal_nan=True)     # an infinity of the weight's sign, NaN for zero
            keep = torch.arange(tokens, device=DEV) != row
            assert torch.equal(y[keep], plain[keep])


@pytest.mark.parametrize("tokens,k", A16)
def test_w4a16_no_overflow_below_the_stated_bound(tokens, k):
    """Activations of one sign with k max |x| = 2^116 against the largest
    weights: the exact sum, 2688 2^116, is the largest partial one."""
    note(f"w4a16 large tokens={tokens} k={k}")
    x = 2.0 ** (116 - int(np.ceil(np.log2(k))))
    out = 40
    p, c = np.full((out, k // 2), 0x77, np.uint8), np.full((out, k // 16), 0x7E, np.uint8)
    y = nq.matmul_w4a16(to_dev_bf16(F.f64_to_bf16_rne(np.full((tokens, k), x))), to_dev_u8(p), to_dev_u8(c),
                        to_dev_f32([2.0 ** -20]))
    _near(_values(y), np.full((tokens, k), x), np.full((out, k), 2688.0), 2.0 ** -20)


# ---------------------------------------------------------------- layer ----

def _e2m1(p):
    """float64 values of packed nibbles, on the GPU."""
    m = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    t = torch.cat((m, -m))
    return torch.stack((t[(p & 15).long()], t[(p >> 4).long()]), -1).flatten(-2)


def _nv(p, c, s2):
    """float64 values of one expert's matrix, on the GPU."""
    v = _e2m1(p).unflatten(-1, (-1, 16)) * c.view(torch.float8_e4m3fn).double()[..., None]
    return v.flatten(-2) * float(s2)


class Experts:
    """Random experts made and kept on the GPU, and their float64 layer."""

    def __init__(self, seed, tokens, hidden, inter, experts, top_k, lo=40, hi=96):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        u8 = lambda a, b, *s: torch.randint(a, b, s, generator=g, device=DEV, dtype=torch.uint8)
        self.dims = (tokens, hidden, inter, experts, top_k)
        self.x = torch.randn((tokens, hidden), generator=g, device=DEV).to(torch.bfloat16)
        # values of about rms: nibbles 2.7, codes up to 2^((hi - 57) / 8)
        rms = 2.7 * 2.0 ** ((hi - 57) / 8 - 1)
        spread = lambda k: (torch.rand(experts, generator=g, device=DEV) + 0.5) / (rms * k ** 0.5)
        self.w = [u8(0, 256, experts, 2, inter, hidden // 2), u8(lo, hi, experts, 2, inter, hidden // 16), spread(hidden),
                  u8(0, 256, experts, hidden, inter // 2), u8(lo, hi, experts, hidden, inter // 16), spread(inter)]
        self.ids = torch.rand((tokens, experts), generator=g, device=DEV).argsort(1)[:, :top_k].int().contiguous()
        self.wt = torch.rand((tokens, top_k), generator=g, device=DEV)

    def run(self):
        return nq.moe_forward(self.x, self.ids, self.wt, *self.w)

    def check(self, y, rows=None):
        """Bounds: each product's sums, the first's carried through silu (slope
        below 1.1), and 2^-20 of silu(gate) up for the exponential and the few
        fp32 operations around it."""
        tokens, hidden, inter, experts, top_k = self.dims
        u = 2.0 ** -23
        rows = torch.arange(tokens, device=DEV) if rows is None else torch.as_tensor(rows, device=DEV)
        x, ids, wt = self.x[rows].double(), self.ids[rows], self.wt[rows].double()
        ref, bound = torch.zeros_like(x), torch.zeros_like(x)
        for e in torch.unique(ids).tolist():
            if not 0 <= e < experts:
                continue
            t = torch.nonzero((ids == e).any(1))[:, 0]
            w13 = _nv(self.w[0][e], self.w[1][e], self.w[2][e])
            gate, up = (x[t] @ w13[i].t() for i in (0, 1))
            eg, eu = ((hidden + 3) * u * (x[t].abs() @ w13[i].abs().t()) for i in (0, 1))
            act = gate * torch.sigmoid(gate)
            h = act * up
            eh = 1.1 * eg * (up.abs() + eu) + act.abs() * eu + 2.0 ** -20 * h.abs()
            w2 = _nv(self.w[3][e], self.w[4][e], self.w[5][e])
            share = (wt[t] * (ids[t] == e)).sum(1, keepdim=True)
            ref.index_add_(0, t, share * (h @ w2.t()))
            bound.index_add_(0, t, share.abs() * (eh * (1 + 2.0 ** -10) @ w2.abs().t() +
                                                  (inter * 2 + top_k + 16) * u * (h.abs() @ w2.abs().t())))
        got = y[rows].double()
        err = (got - ref).abs()
        assert bool((err <= bound * (1 + HALF) + HALF * ref.abs() + 1e-38).all())
        assert float((got - ref).norm()) <= HALF * float(ref.norm())


@pytest.mark.parametrize("tokens", [1, 16, 61, 64])
@pytest.mark.parametrize("hidden,inter", [(528, 1040), (1024, 1552), (272, 2048), (512, 4112)])
def test_layer_long_inter(tokens, hidden, inter):
    """Experts of three and more quads of channels."""
    note(f"layer tokens={tokens} hidden={hidden} inter={inter}")
    L = Experts(tokens + inter, tokens, hidden, inter, 12, 3)
    L.check(L.run())


@pytest.mark.parametrize("tokens", [1, 5, 16, 61, 64])
def test_layer_full_size(tokens):
    """128 experts of 2048 x 7168, eight a token."""
    note(f"layer full size tokens={tokens}")
    L = Experts(tokens, tokens, 7168, 2048, 128, 8)
    L.check(L.run(), sorted({0, tokens // 3, tokens // 2, tokens - 1}))


@pytest.mark.parametrize("tokens", [2, 40])
def test_layer_experts_beyond_32_bit_offsets(tokens):
    """4.8 GB of first and 2.4 GB of second weights; the last experts."""
    note(f"layer 7 GB of weights tokens={tokens}")
    L = Experts(tokens, tokens, 4608, 1024, 1024, 4)
    L.ids = 1023 - L.ids % 40
    L.ids[0] = torch.tensor([1023, 1022, 0, 911], device=DEV)
    L.check(L.run(), range(min(tokens, 8)))


@pytest.mark.parametrize("tokens", [3, 30])
@pytest.mark.parametrize("lo,hi", [(0, 127), (0, 8), (0x78, 0x7F)])
def test_layer_codes_of_the_whole_range(tokens, lo, hi):
    note(f"layer codes {lo}..{hi - 1} tokens={tokens}")
    L = Experts(tokens + hi, tokens, 272, 160, 6, 3, lo, hi)
    L.check(L.run())


@pytest.mark.parametrize("tokens", [3, 30])
def test_layer_gates_far_from_zero(tokens):
    """silu at both ends: gates of hundreds."""
    note(f"layer large gates tokens={tokens}")
    L = Experts(tokens, tokens, 272, 160, 6, 3)
    L.w[2] = L.w[2] * 300.0
    L.check(L.run())


@pytest.mark.parametrize("tokens", [4, 24])
def test_layer_nan_and_infinite_tokens_and_weights(tokens):
    """They reach the outputs of their own token alone."""
    note(f"layer nan tokens={tokens}")
    L = Experts(tokens, tokens, 256, 96, 5, 2)
    plain = L.run().clone()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for which in ("x", "wt"):
            t = getattr(L, which)
            keep = t[2, 1].clone()
            t[2, 1] = bad
            y = L.run()
            rows = torch.arange(tokens, device=DEV) != 2
            assert torch.equal(y[rows], plain[rows])
            assert not bool(torch.isfinite(y[2]).any())
            t[2, 1] = keep
