"""GPU parity of the MXFP4 quantizer, the packed 4-bit products and the expert
layer against the float64 oracle.

Bounds.  Operands and products are exact, so an output differs from the exact
sum by the fp32 accumulation (every addition at most one unit in the last
place, 2^-23, of a partial sum that the sum of magnitudes bounds: k 2^-23 of
it, and 3 more for the tensor scales and partial tiles) and by one rounding to
bf16 (half a step, 2^-8 of the value).  The layer's bound carries the first
product's through silu (slope below 1.1) and adds the two-part bf16 form of
silu * up (2^-16 of it) and 2^-20 for the exponential and the few fp32
operations around it."""
import numpy as np
import pytest
import torch

import datagen
import oracle as O
from oracle import formats as F
from oracle import mxcast as M
import nvfp4_post_quantization_amd as nq

from _gpu import DEV, need_gpu, note, to_dev_bf16, to_dev_f32, to_dev_u8, host, to_host_bits

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8           # half a bf16 step, relative


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _laplace(rng, rows, k, b=1.0):
    return datagen.f32_to_bf16_bits(rng.laplace(0, b, (rows, k)).astype(np.float32))


def _strided(bits, ld):
    full = np.full((bits.shape[0], ld), 0x7FC0, np.uint16)          # NaN around the matrix
    full[:, :bits.shape[1]] = bits
    return to_dev_bf16(full)[:, :bits.shape[1]]


# ------------------------------------------------------------ quantizer ----

@pytest.mark.parametrize("rows,k,ld", [(1, 32, 32), (3, 64, 64), (5, 96, 104), (333, 288, 288), (64, 4096, 4096),
                                       (1000, 1024, 1032), (2, 12288, 12288), (4097, 160, 168)])
def test_quantize_and_dequant(rows, k, ld):
    note(f"mxfp4 quantize rows={rows} k={k} ld={ld}")
    rng = np.random.default_rng(rows * 7 + k)
    bits = _laplace(rng, rows, k) if rows != 64 else _laplace(rng, rows, k, 1e-37)
    bits[0, :7] = 0x8000, 0x0001, 0x807F, 0x0080, 0x3F80, 0x40E0, 0xC0A0
    p, e = nq.mxfp4_quantize(_strided(bits, ld))
    pr, er = O.mxfp4_quantize(bits)
    assert np.array_equal(host(e), er) and np.array_equal(host(p), pr)
    got = to_host_bits(nq.mxfp4_dequant(p, e))
    assert np.array_equal(got, F.f64_to_bf16_rne(M.mxfp4_dequant(pr, er)))


def test_quantize_every_bf16_in_blocks_of_every_scale():
    """Blocks [peak, 31 smaller values]: every finite bf16 magnitude occurs
    under its own binade's scale and under larger ones."""
    note("mxfp4 quantize exhaustive")
    pat = np.arange(0x7F80, dtype=np.uint16)
    out = []
    for up in (0, 1, 2, 3, 5, 40):
        peak = np.minimum((pat.astype(np.int64) | 0x7F) + 128 * up, 0x7F7F).astype(np.uint16)
        b = np.repeat(pat[:, None], 32, 1)
        b[:, 1::2] |= 0x8000
        b[:, 5] = peak
        out.append(b)
    bits = np.concatenate(out)
    p, e = nq.mxfp4_quantize(to_dev_bf16(bits))
    pr, er = O.mxfp4_quantize(bits)
    assert np.array_equal(host(e), er) and np.array_equal(host(p), pr)


def test_quantize_zero_and_nonfinite_blocks():
    note("mxfp4 quantize edges")
    bits = np.zeros((8, 64), np.uint16)
    bits[1, 3], bits[2, 40], bits[3, 63], bits[4, 32] = 0x7F80, 0x7FC1, 0xFF80, 0xFF81
    bits[1:5, 10] = 0x3F80
    bits[5] = 0x8000
    bits[6, ::5] = 0x7F7F
    p, e = nq.mxfp4_quantize(to_dev_bf16(bits))
    pr, er = O.mxfp4_quantize(bits)
    assert np.array_equal(host(e), er) and np.array_equal(host(p), pr)
    v = F.bf16_bits_to_f64(to_host_bits(nq.mxfp4_dequant(p, e)))
    assert np.array_equal(np.isnan(v), np.repeat(er == 255, 32, 1))


def test_dequant_all_codes():
    note("mxfp4 dequant all codes")
    p = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    p = np.tile(p, (1, 16)).reshape(256, 256)
    e = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))
    got = to_host_bits(nq.mxfp4_dequant(to_dev_u8(p), to_dev_u8(e)))
    v = M.mxfp4_dequant(p, e)
    nan = np.isnan(v)
    assert np.array_equal(got[~nan], F.f64_to_bf16_rne(v[~nan])) and np.all((got[nan] & 0x7FFF) > 0x7F80)


def test_quantize_beyond_32_bit_offsets():
    note("mxfp4 quantize 600000 x 4096")
    rows, k = 600_000, 4096                                           # 4.9 GB of bf16
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device=DEV)
    bits = _laplace(np.random.default_rng(1), 40, k)
    x[-40:] = to_dev_bf16(bits)
    p, e = nq.mxfp4_quantize(x)
    pr, er = O.mxfp4_quantize(bits)
    assert np.array_equal(host(e[-40:]), er) and np.array_equal(host(p[-40:]), pr)
    assert int(p[:-40].max()) == 0 and int(e[:-40].max()) == 0
    assert np.array_equal(to_host_bits(nq.mxfp4_dequant(p, e)[-40:]), F.f64_to_bf16_rne(M.mxfp4_dequant(pr, er)))


# ------------------------------------------------------------- products ----

def _nv(rng, rows, k, lo=0, hi=127):
    p = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    c = rng.integers(lo, hi, (rows, k // 16), dtype=np.uint8)
    return p, c, float(np.float32(rng.random() * 0.01 + 1e-4))


def _mx(rng, rows, k):
    return rng.integers(0, 256, (rows, k // 2), dtype=np.uint8), rng.integers(118, 134, (rows, k // 32), dtype=np.uint8)


class Case:
    """Inputs of one product, its exact values and its call."""

    def __init__(self, kind, rng, tokens, out, k, ldx=None):
        self.kind, self.shape = kind, (tokens, out, k)
        if kind == "mx":
            x, w = _mx(rng, tokens, k), _mx(rng, out, k)
            self.x, self.w = M.mxfp4_dequant(*x), M.mxfp4_dequant(*w)
            self.args = [to_dev_u8(a) for a in (*x, *w)]
        else:
            w = _nv(rng, out, k)
            self.w = O.nvfp4_values(*w)
            wd = [to_dev_u8(w[0]), to_dev_u8(w[1]), to_dev_f32([w[2]])]
            if kind == "w4a16":
                bits = _laplace(rng, tokens, k)
                self.x = F.bf16_bits_to_f64(bits)
                self.args = [_strided(bits, ldx or k)] + wd
            else:
                x = _nv(rng, tokens, k)
                self.x = O.nvfp4_values(*x)
                self.args = [to_dev_u8(x[0]), to_dev_u8(x[1]), to_dev_f32([x[2]])] + wd
        self.fn = {"mx": nq.mxfp4_matmul, "w4a16": nq.matmul_w4a16, "w4a4": nq.matmul_w4a4}[kind]
        q = nq.mxfp4_matmul_workspace_bytes if kind == "mx" else nq.matmul_workspace_bytes
        self.ws_bytes = q(tokens, out, k)

    def workspace(self, fill):
        return torch.full((max(self.ws_bytes, 1),), fill, dtype=torch.uint8, device=DEV)

    def check(self, y, rows=slice(None)):
        ref, mag = O.matmul(self.x[rows], self.w)
        got = F.bf16_bits_to_f64(to_host_bits(y[rows]))
        bound = HALF * np.abs(ref) + (self.shape[2] + 3) * 2.0 ** -23 * mag * (1 + HALF) + 1e-38
        err = np.abs(got - ref)
        assert np.all(err <= bound), f"max excess {np.max(err / bound):.3f} at {np.argwhere(err > bound)[:4].tolist()}"
        assert np.linalg.norm(got - ref) <= HALF * np.linalg.norm(ref)


KINDS = ["mx", "w4a16", "w4a4"]
# tokens, out, k, x row stride beyond k, y row stride beyond out.  k: shorter
# than a block group, ending inside one, long; tokens and rows around every
# tile size; strides that leave rows unaligned.
SHAPES = [
    (1, 1, 32, 0, 0), (1, 16, 64, 0, 0), (2, 17, 96, 8, 1), (3, 5, 128, 0, 3), (5, 64, 160, 8, 0), (16, 33, 256, 0, 7),
    (17, 48, 288, 16, 0), (31, 100, 512, 0, 4), (33, 127, 544, 0, 1), (64, 128, 1024, 0, 0), (65, 129, 992, 8, 3),
    (100, 256, 2048, 0, 0), (128, 200, 4064, 0, 8), (129, 257, 384, 0, 0), (255, 512, 640, 24, 0), (300, 300, 1312, 0, 5),
    (513, 130, 224, 0, 2), (1, 2048, 12288, 0, 0), (7, 515, 4128, 0, 0), (256, 256, 32, 0, 0), (260, 1040, 608, 8, 0),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,out,k,px,py", SHAPES)
def test_product(kind, tokens, out, k, px, py):
    note(f"{kind} tokens={tokens} out={out} k={k} ldx+{px} ldy+{py}")
    c = Case(kind, np.random.default_rng(tokens * 31 + out * 7 + k), tokens, out, k, k + px)
    ld = out + py
    buf = torch.full((tokens + 2, ld), 7.0, dtype=torch.bfloat16, device=DEV)
    y = buf[1:-1, :out]
    assert c.fn(*c.args, out=y, workspace=c.workspace(0xFF)) is y
    c.check(y)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all()) and bool((buf[:, out:] == 7).all())
    again = c.fn(*c.args, workspace=c.workspace(0x3C))                # whatever the workspace held
    assert torch.equal(again.view(torch.int16), y.contiguous().view(torch.int16))


@pytest.mark.parametrize("kind", ["w4a16", "w4a4"])
@pytest.mark.parametrize("tokens,out,k", [(1, 8, 16), (4, 40, 48), (20, 33, 80), (70, 70, 144), (130, 260, 272),
                                          (257, 513, 1040), (66, 128, 2064)])
def test_product_half_chunk_rows(kind, tokens, out, k):
    """k an odd multiple of 16: rows of packed nibbles that are only 8-byte
    aligned and of codes at odd addresses."""
    note(f"{kind} tokens={tokens} out={out} k={k}")
    c = Case(kind, np.random.default_rng(tokens + out + k), tokens, out, k)
    c.check(c.fn(*c.args, workspace=c.workspace(0xFF)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [3, 6, 12, 16, 24])
def test_product_few_tokens_many_channels(kind, tokens):
    """More channels than the waves of a workgroup hold at a time, the last
    ones a part of a wave's share."""
    for out, k in ((70, 12320), (33, 8224), (4100, 8704)):
        note(f"{kind} tokens={tokens} out={out} k={k}")
        c = Case(kind, np.random.default_rng(tokens + out), tokens, out, k)
        c.check(c.fn(*c.args, workspace=c.workspace(0xFF)))
    if kind != "mx":
        note(f"{kind} tokens={tokens} k=8208")
        c = Case(kind, np.random.default_rng(tokens), tokens, 90, 8208)
        c.check(c.fn(*c.args, workspace=c.workspace(0xFF)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,out,k", [(300, 13000, 320), (300, 13000, 416), (130, 140, 4992), (70, 260, 20000),
                                          (40, 1000, 128), (200, 2050, 1152)])
def test_product_small_tiles(kind, tokens, out, k):
    """Tiles that share a CU, and channels split into parts of unequal length."""
    note(f"{kind} tokens={tokens} out={out} k={k}")
    c = Case(kind, np.random.default_rng(tokens + k), tokens, out, k)
    c.check(c.fn(*c.args, workspace=c.workspace(0xFF)))


@pytest.mark.parametrize("kind", KINDS)
def test_product_two_streams(kind):
    note(f"{kind} two streams")
    a, b = (Case(kind, np.random.default_rng(i), t, 2000, 2048) for i, t in ((1, 5), (2, 150)))
    want = [c.fn(*c.args).clone() for c in (a, b)]
    ws = [c.workspace(0xFF) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for c, w, s in zip((a, b), ws, streams):
            with torch.cuda.stream(s):
                got.append(c.fn(*c.args, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("kind", KINDS)
def test_product_no_tokens(kind):
    note(f"{kind} no tokens")
    c = Case(kind, np.random.default_rng(0), 1, 16, 64)
    empty = [a[:0] if i < (1 if kind == "w4a16" else 2) else a for i, a in enumerate(c.args)]
    assert c.fn(*empty).shape == (0, 16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [3, 70, 300])
def test_product_nan_scales_stay_in_their_row(kind, tokens):
    note(f"{kind} nan scales tokens={tokens}")
    c = Case(kind, np.random.default_rng(tokens), tokens, 140, 320)
    plain = c.fn(*c.args).clone()
    nan = 255 if kind == "mx" else 0x7F
    w_scales = c.args[3] if kind == "mx" else c.args[2] if kind == "w4a16" else c.args[4]
    w_scales[131, -1] = nan
    y = c.fn(*c.args)
    assert bool(torch.isnan(y[:, 131]).all())
    keep = torch.ones(140, dtype=torch.bool, device=DEV)
    keep[131] = False
    assert torch.equal(y[:, keep], plain[:, keep])
    if kind != "w4a16":
        c.args[1][2, 0] = nan
        y = c.fn(*c.args)
        assert bool(torch.isnan(y[2]).all())
        rows = torch.ones(tokens, dtype=torch.bool, device=DEV)
        rows[2] = False
        assert torch.equal(y[rows][:, keep], plain[rows][:, keep])


@pytest.mark.parametrize("kind", KINDS)
def test_product_full_size_sampled(kind):
    """Gate projection over a prompt batch and down projection over a short
    ragged one, sampled rows against the oracle."""
    for tokens, out, k in ((2048, 12288, 4096), (333, 4096, 12288), (2049, 6200, 160), (3333, 4100, 608)):
        note(f"{kind} tokens={tokens} out={out} k={k}")
        c = Case(kind, np.random.default_rng(k), tokens, out, k)
        y = c.fn(*c.args, workspace=c.workspace(0xFF))
        rows = np.r_[0, 1, tokens - 1, np.random.default_rng(1).choice(tokens, 13, replace=False)]
        c.check(y, rows)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [2, 70])
def test_product_weights_beyond_32_bit_offsets(kind, tokens):
    """Packed weights of 4.3 GB: the last output rows."""
    note(f"{kind} 4.3 GB of weights tokens={tokens}")
    out, k, tail = 1_050_000, 8192, 32
    c = Case(kind, np.random.default_rng(9), tokens, tail, k)
    n = len(c.args) - (2 if kind == "mx" else 3)
    big = []
    for i, a in enumerate(c.args):
        if i >= n and a.dim() == 2:
            b = torch.zeros((out, a.shape[1]), dtype=a.dtype, device=DEV)
            b[-tail:] = a
            a = b
        big.append(a)
    y = c.fn(*big)
    c.check(y[:, -tail:].contiguous())
    assert float(y[:, :-tail].abs().max()) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_product_output_beyond_32_bit_offsets(kind):
    note(f"{kind} output rows 5 GB apart")
    tokens, out, k, ld = 300, 24, 64, 8_400_000
    c = Case(kind, np.random.default_rng(10), tokens, out, k)
    buf = torch.zeros((tokens, ld), dtype=torch.bfloat16, device=DEV)
    c.check(c.fn(*c.args, out=buf[:, :out]))
    assert float(buf[:, out].abs().max()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [4, 200])
def test_product_stream_and_graph(kind, tokens):
    """Eager on a side stream, then captured: each replay follows new inputs,
    with eager work in between."""
    note(f"{kind} stream and graph tokens={tokens}")
    rng = np.random.default_rng(tokens)
    cases = [Case(kind, rng, tokens, 160, 2080) for _ in range(3)]
    want = [c.fn(*c.args).clone() for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cases[0].fn(*cases[0].args)
    side.synchronize()
    assert torch.equal(got, want[0])
    static = [a.clone() for a in cases[0].args]
    y = torch.empty((tokens, 160), dtype=torch.bfloat16, device=DEV)
    ws = cases[0].workspace(0xFF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cases[0].fn(*static, out=y, workspace=ws)
    for i in (1, 2, 0, 2):
        for s, a in zip(static, cases[i].args):
            s.copy_(a)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        cases[i].check(cases[i].fn(*cases[i].args))


@pytest.mark.parametrize("kind", KINDS)
def test_product_refuses_what_does_not_fit(kind):
    note(f"{kind} refusals")
    c = Case(kind, np.random.default_rng(0), 4, 32, 64)
    with pytest.raises(ValueError):
        c.fn(*c.args, out=torch.empty((4, 31), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        c.fn(*c.args, out=torch.empty((4, 32), dtype=torch.float32, device=DEV))
    with pytest.raises(ValueError):
        c.fn(*c.args, out=torch.empty((32, 4), dtype=torch.bfloat16, device=DEV).t())
    bad = list(c.args)
    bad[-1 if kind == "mx" else -2] = bad[-1 if kind == "mx" else -2][:, :-1]
    with pytest.raises(ValueError):
        c.fn(*bad)
    with pytest.raises(ValueError):
        c.fn(c.args[0].cpu(), *c.args[1:])


# ---------------------------------------------------------------- layer ----

class Layer:
    def __init__(self, rng, tokens, hidden, inter, experts, top_k, ldx=0):
        self.dims = (tokens, hidden, inter, experts, top_k)
        self.xb = datagen.f32_to_bf16_bits(rng.normal(0, 1, (tokens, hidden)).astype(np.float32))
        self.x = F.bf16_bits_to_f64(self.xb)
        p13, c13 = (rng.integers(0, 256, (experts, 2, inter, hidden // 2), dtype=np.uint8),
                    rng.integers(40, 96, (experts, 2, inter, hidden // 16), dtype=np.uint8))
        p2, c2 = (rng.integers(0, 256, (experts, 1, hidden, inter // 2), dtype=np.uint8),
                  rng.integers(40, 96, (experts, 1, hidden, inter // 16), dtype=np.uint8))
        s13 = (rng.random(experts) + 0.5).astype(np.float32) * np.float32(0.1 / np.sqrt(hidden))
        s2 = (rng.random(experts) + 0.5).astype(np.float32) * np.float32(0.1 / np.sqrt(inter))
        self.ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]).astype(np.int32)
        self.wt = rng.random((tokens, top_k)).astype(np.float32)
        self.w13, self.w2 = O.nvfp4_values(p13, c13, s13), O.nvfp4_values(p2, c2, s2)[:, 0]
        self.xd = _strided(self.xb, hidden + ldx)
        self.weights = [to_dev_u8(p13), to_dev_u8(c13), to_dev_f32(s13), to_dev_u8(p2), to_dev_u8(c2), to_dev_f32(s2)]

    def workspace(self, fill):
        n = nq.moe_workspace_bytes(self.dims[0], self.dims[4], self.dims[2])
        return torch.full((n,), fill, dtype=torch.uint8, device=DEV)

    def routing(self):
        return torch.from_numpy(self.ids).to(DEV), to_dev_f32(self.wt)

    def run(self, **kw):
        return nq.moe_forward(self.xd, *self.routing(), *self.weights, **kw)

    def check(self, y):
        tokens, hidden, inter, experts, top_k = self.dims
        ref, bound = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
        u = 2.0 ** -23
        for t in range(tokens):
            for s in range(top_k):
                e = int(self.ids[t, s])
                if not 0 <= e < experts:
                    continue
                gate, up = self.w13[e] @ self.x[t]
                eg, eu = (hidden + 3) * u * (np.abs(self.w13[e]) @ np.abs(self.x[t]))
                act = gate / (1 + np.exp(-gate))
                h = act * up
                eh = 1.1 * eg * (np.abs(up) + eu) + np.abs(act) * eu + (2.0 ** -16 + 2.0 ** -20) * np.abs(h)
                a = np.abs(self.w2[e])
                w = abs(float(self.wt[t, s]))
                ref[t] += float(self.wt[t, s]) * (self.w2[e] @ h)
                bound[t] += w * (a @ (eh * (1 + 2.0 ** -10)) + (inter * 2 + top_k + 16) * u * (a @ np.abs(h)))
        got = F.bf16_bits_to_f64(to_host_bits(y))
        bound = bound * (1 + HALF) + HALF * np.abs(ref) + 1e-38
        err = np.abs(got - ref)
        assert np.all(err <= bound), f"max excess {np.max(err / bound):.3f}"
        assert np.linalg.norm(got - ref) <= HALF * np.linalg.norm(ref) or not ref.any()


LAYERS = [(1, 32, 16, 4, 1, 0), (1, 128, 128, 8, 2, 0), (2, 48, 80, 5, 5, 8), (3, 272, 144, 16, 4, 0), (7, 256, 96, 3, 2, 8),
          (16, 512, 272, 32, 8, 0), (17, 160, 64, 4, 2, 0), (33, 320, 160, 9, 3, 0), (40, 144, 48, 2, 2, 0),
          (64, 256, 128, 128, 8, 0), (64, 96, 32, 1, 1, 0), (5, 64, 32, 1024, 16, 0), (61, 1040, 400, 64, 6, 8)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,px", LAYERS)
def test_layer(tokens, hidden, inter, experts, top_k, px):
    note(f"moe tokens={tokens} hidden={hidden} inter={inter} experts={experts} top_k={top_k}")
    L = Layer(np.random.default_rng(tokens * 3 + hidden + experts), tokens, hidden, inter, experts, top_k, px)
    buf = torch.full((tokens + 2, hidden + 3), 5.0, dtype=torch.bfloat16, device=DEV)
    y = buf[1:-1, :hidden]
    L.run(out=y, workspace=L.workspace(0xFF))
    L.check(y)
    assert bool((buf[0] == 5).all()) and bool((buf[-1] == 5).all()) and bool((buf[:, hidden:] == 5).all())
    again = L.run(workspace=L.workspace(0x3C))
    assert torch.equal(again.view(torch.int16), y.contiguous().view(torch.int16))


# Every number of output rows a workgroup takes, and more channels than the
# waves of a workgroup hold at a time.
@pytest.mark.parametrize("hidden,inter", [(4112, 48), (5152, 32), (6160, 544), (7184, 32), (8704, 32), (9232, 16)])
def test_layer_wide(hidden, inter):
    for tokens in (2, 5):
        note(f"moe tokens={tokens} hidden={hidden} inter={inter}")
        L = Layer(np.random.default_rng(hidden + tokens), tokens, hidden, inter, 3, 2)
        L.check(L.run(workspace=L.workspace(0xFF)))


@pytest.mark.parametrize("tokens", [4, 20, 64])
def test_layer_empty_places_foreign_ids_and_repeats(tokens):
    note(f"moe odd ids tokens={tokens}")
    L = Layer(np.random.default_rng(tokens), tokens, 160, 96, 6, 4)
    L.ids[0] = -1                                                     # nothing at all
    L.ids[1] = 3, 3, 3, 1                                             # the same expert three times
    L.ids[2] = 2, -1, 6, 2 ** 31 - 1                                  # outside the experts
    L.ids[3] = -2 ** 31, 0, 0, 5
    if tokens > 40:
        L.ids[4:60] = 4, 5, -1, -1                                    # many tokens on one expert
    y = L.run(workspace=L.workspace(0xFF))
    L.check(y)
    assert float(y[0].abs().max()) == 0
    L.ids[:] = -1
    assert float(L.run(workspace=L.workspace(0xFF)).abs().max()) == 0


def test_layer_nan_expert_reaches_its_tokens_only():
    note("moe nan expert")
    L = Layer(np.random.default_rng(2), 24, 128, 64, 6, 2)
    plain = L.run().clone()
    served = torch.from_numpy((L.ids == 3).any(1)).to(DEV)
    assert bool(served.any()) and not bool(served.all())
    for which, at in ((1, (3, 0, 5, 2)), (4, (3, 0, 7, 1))):
        keep = int(L.weights[which][at])
        L.weights[which][at] = 0x7F
        y = L.run()
        assert bool(torch.isnan(y[served]).any(1).all()) and torch.equal(y[~served], plain[~served])
        L.weights[which][at] = keep


def test_layer_no_tokens_and_refusals():
    note("moe refusals")
    L = Layer(np.random.default_rng(3), 2, 64, 32, 4, 2)
    i, w = L.routing()
    assert nq.moe_forward(L.xd[:0], i[:0], w[:0], *L.weights).shape == (0, 64)
    with pytest.raises(nq.NvFp4Error) as e:
        nq.moe_forward(torch.zeros((65, 64), dtype=torch.bfloat16, device=DEV), i[:1].expand(65, 2).contiguous(),
                       w[:1].expand(65, 2).contiguous(), *L.weights)
    assert e.value.status == 5
    with pytest.raises(nq.NvFp4Error) as e:
        nq.moe_forward(L.xd, i, w, *L.weights, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4
    with pytest.raises(TypeError):
        nq.moe_forward(L.xd, i.long(), w, *L.weights)
    with pytest.raises(ValueError):
        nq.moe_forward(L.xd, i, w[:1], *L.weights)
    with pytest.raises(ValueError):
        nq.moe_forward(L.xd, i, w, *L.weights[:3], L.weights[3][:, :, :-1], *L.weights[4:])


def test_layer_graph():
    note("moe graph")
    rng = np.random.default_rng(4)
    L = [Layer(rng, 12, 256, 160, 16, 4) for _ in range(3)]
    want = [l.run().clone() for l in L]
    static = [L[0].xd.clone(), *L[0].routing(), *[a.clone() for a in L[0].weights]]
    y = torch.empty((12, 256), dtype=torch.bfloat16, device=DEV)
    ws = L[0].workspace(0xFF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nq.moe_forward(*static, out=y, workspace=ws)
    for i in (1, 0, 2, 1):
        for s, a in zip(static, [L[i].xd, *L[i].routing(), *L[i].weights]):
            s.copy_(a)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(L[i].run(), want[i])


@pytest.mark.parametrize("tokens,experts,top_k,normalize", [(1, 1, 1, True), (3, 5, 5, False), (64, 64, 6, True),
                                                            (130, 65, 8, True), (9, 128, 8, False), (33, 256, 16, True),
                                                            (1000, 1000, 4, False), (2, 1024, 16, True)])
def test_route(tokens, experts, top_k, normalize):
    note(f"route tokens={tokens} experts={experts} top_k={top_k}")
    rng = np.random.default_rng(experts + tokens)
    z = rng.normal(0, 2, (tokens, experts)).astype(np.float32)
    z[:, ::3] = np.round(z[:, ::3])                                   # ties
    z[0, 0] = np.inf
    if tokens > 2:
        z[1, experts // 2:] = np.nan
        z[2] = -np.inf
    full = np.full((tokens, experts + 3), 1e30, np.float32)
    full[:, :experts] = z
    ids, w = nq.moe_route(torch.from_numpy(full).to(DEV)[:, :experts], top_k, normalize=normalize)
    ri, rw = O.moe_route(z, top_k, normalize)
    assert np.array_equal(host(ids), ri)
    # the difference of two logits, one exponential (2 units in the last place
    # each with its argument's rounding of up to |z| 2^-24), a sum, a quotient
    tol = (64 + experts) * 2.0 ** -24
    assert np.all(np.abs(host(w) - rw) <= tol * rw + 1e-37)


# --------------------------------------------------------- used together ----

def test_calibrated_linear_run():
    """A Linear as it is calibrated and then used: Hessian, sweep, W4A16 and
    W4A4 products of the packed weight."""
    note("calibrated linear")
    w, x = datagen.config1()
    wd, xd = to_dev_bf16(w), to_dev_bf16(x)
    s2, _ = nq.compute_scale2(wd)
    H = torch.zeros((16, 16, 16), dtype=torch.float32, device=DEV)
    nq.hessian_accum(xd, H)
    p, c, _ = nq.scale_sweep(wd, H, s2)
    wv = O.nvfp4_values(host(p), host(c), float(s2))
    xv = F.bf16_bits_to_f64(x)
    k = xv.shape[1]
    def near(y, xv):
        ref, mag = O.matmul(xv, wv)
        assert np.all(np.abs(F.bf16_bits_to_f64(to_host_bits(y)) - ref) <=
                      HALF * np.abs(ref) + (k + 3) * 2.0 ** -23 * mag * (1 + HALF))
        return ref
    y = near(nq.matmul_w4a16(xd, p, c, s2), xv)
    full = xv @ F.bf16_bits_to_f64(w).T
    assert np.linalg.norm(y - full) < 0.2 * np.linalg.norm(full)
    s2x, _ = nq.compute_scale2(xd)
    q, qc = nq.quantize_dynamic(xd, s2x)
    near(nq.matmul_w4a4(q, qc, s2x, p, c, s2), O.nvfp4_values(host(q), host(qc), float(s2x)))
    mw, mx = nq.mxfp4_quantize(wd), nq.mxfp4_quantize(xd)
    wv = M.mxfp4_dequant(*[host(a) for a in mw])
    near(nq.mxfp4_matmul(*mx, *mw), M.mxfp4_dequant(*[host(a) for a in mx]))


def test_cast_experts_run():
    """Experts quantized to MXFP4, cast to NVFP4, routed and run."""
    note("cast experts")
    rng = np.random.default_rng(8)
    tokens, hidden, inter, experts, top_k = 6, 128, 64, 8, 2
    def cast(mats, rows, k):
        bits = datagen.f32_to_bf16_bits(rng.normal(0, 0.05, (experts * mats * rows, k)).astype(np.float32))
        p, e = nq.mxfp4_quantize(to_dev_bf16(bits))
        p, e = p.view(experts, mats, rows, k // 2), e.view(experts, mats, rows, k // 32)
        before = M.mxfp4_dequant(host(p).copy(), host(e))
        c, s2, fb = nq.mxfp4_to_nvfp4_cast(p, e)
        assert int(fb.sum()) == 0
        assert np.array_equal(O.nvfp4_values(host(p), host(c), host(s2)), before)
        return p, c, s2
    w13, w2 = cast(2, inter, hidden), cast(1, hidden, inter)
    L = Layer(rng, tokens, hidden, inter, experts, top_k)
    L.weights = [*w13, *w2]
    L.w13 = O.nvfp4_values(*[host(a) for a in w13])
    L.w2 = O.nvfp4_values(*[host(a) for a in w2])[:, 0]
    logits = rng.normal(0, 1, (tokens, experts)).astype(np.float32)
    ids, wts = nq.moe_route(torch.from_numpy(logits).to(DEV), top_k)
    L.ids, L.wt = host(ids), host(wts)
    L.check(nq.moe_forward(L.xd, ids, wts, *L.weights))
