"""W4A16 products with low-rank adapters against float64: sums of n products in
fp32 are off by n 2^-23 of the sum of magnitudes, the result by half a bf16 step
more, 2^-8 of its value."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
import oracle as O
from oracle import formats as F
from oracle import layer as L

from _gpu import DEV, need_gpu, note, to_dev_bf16, to_dev_f32, to_dev_u8, to_host_bits

pytestmark = pytest.mark.gpu

HALF, EPS = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


class Case:
    def __init__(self, seed, tokens, out, k, adapters, rank, ids="any"):
        rng = np.random.default_rng(seed)
        self.dims = tokens, out, k, rank
        self.x = F.f64_to_bf16_bits(rng.standard_normal((tokens, k)))
        self.p = rng.integers(0, 256, (out, k // 2), dtype=np.uint8)
        self.c = rng.integers(0, 0x50, (out, k // 16), dtype=np.uint8)
        self.s2 = np.float32(0.01)
        self.a = F.f64_to_bf16_bits(rng.standard_normal((adapters, rank, k)) / np.sqrt(k))
        self.b = F.f64_to_bf16_bits(rng.standard_normal((adapters, out, rank)))
        self.scale = rng.standard_normal(adapters).astype(np.float32)
        if ids == "any":
            self.ids = rng.integers(-1, adapters + 1, tokens)
        elif ids == "runs":
            self.ids = np.sort(rng.integers(0, adapters, tokens))
        else:
            self.ids = np.full(tokens, ids)
        self.ids = self.ids.astype(np.int32)

    def args(self):
        return [to_dev_u8(self.p), to_dev_u8(self.c), to_dev_f32([self.s2]), torch.from_numpy(self.ids).to(DEV),
                to_dev_bf16(self.a), to_dev_bf16(self.b), to_dev_f32(self.scale)]

    def run(self, x=None, out=None, ws=None):
        if ws is None:
            ws = torch.full((nq.matmul_lora_workspace_bytes(*self.dims),), 255, dtype=torch.uint8, device=DEV)
        return nq.matmul_w4a16_lora(to_dev_bf16(self.x) if x is None else x, *self.args(), out=out, workspace=ws)

    def check(self, y, tokens=slice(None)):
        x, a, b = (F.bf16_bits_to_f64(v) for v in (self.x, self.a, self.b))
        ref, off = L.matmul_lora(x, O.nvfp4_values(self.p, self.c, float(self.s2)), self.ids, a, b,
                                 self.scale.astype(np.float64), EPS)
        got = F.bf16_bits_to_f64(to_host_bits(y))
        bound = HALF * np.abs(ref) + off * (1 + HALF) + 2.0 ** -120
        assert np.all(np.abs(got - ref)[tokens] <= bound[tokens]), f"{np.nanmax((np.abs(got - ref) / bound)[tokens]):.3f} of the bound"


# tokens x outputs x channels: the streaming kernels of 4, 8, 16 tokens, k off 32; small tiles whole and split, k
# off 64; outputs off 4, 16, 32
SIZES = [(1, 128, 512, 4, 16), (3, 150, 528, 3, 8), (6, 96, 544, 9, 24), (16, 260, 1024, 16, 16), (13, 101, 528, 5, 64),
         (16, 64, 16, 2, 8), (17, 130, 512, 7, 16), (40, 67, 528, 40, 40), (100, 256, 4096, 3, 128), (129, 96, 2064, 4, 256),
         (333, 200, 512, 5, 72), (1, 3, 4096, 1, 256), (1100, 96, 144, 6, 16), (1500, 130, 272, 70, 48)]


@pytest.mark.parametrize("ids", ["any", "runs"])
@pytest.mark.parametrize("tokens,out,k,adapters,rank", SIZES)
def test_product(tokens, out, k, adapters, rank, ids):
    note(f"lora {tokens} tokens {out}x{k}, {adapters} of rank {rank}, {ids}")
    c = Case(tokens + out, tokens, out, k, adapters, rank, ids)
    c.check(c.run())


def test_large_tiles():
    """4096 tokens in 256-row tiles, requests of uneven length."""
    note("lora large tiles")
    c = Case(11, 4096, 4096, 144, 9, 24, "runs")
    c.check(c.run())


@pytest.mark.parametrize("tokens", [5, 60, 400])
def test_tokens_without_adapters_are_the_plain_product(tokens):
    note(f"lora none, {tokens} tokens")
    c = Case(tokens, tokens, 160, 512, 2, 16, -1)
    plain = nq.matmul_w4a16(to_dev_bf16(c.x), *c.args()[:3])
    assert torch.equal(c.run(), plain)
    c.ids[:] = np.where(np.arange(tokens) % 2, 2 ** 31 - 1, -2 ** 31)
    assert torch.equal(c.run(), plain)


@pytest.mark.parametrize("tokens", [4, 80])
def test_no_adapters_at_all(tokens):
    note(f"lora of no adapters, {tokens} tokens")
    c = Case(tokens, tokens, 64, 128, 1, 8, 0)
    c.a, c.b, c.scale = c.a[:0], c.b[:0], c.scale[:0]
    assert torch.equal(c.run(), nq.matmul_w4a16(to_dev_bf16(c.x), *c.args()[:3]))


@pytest.mark.parametrize("tokens", [8, 50, 300])
def test_an_adapter_s_infinities_stay_with_its_tokens(tokens):
    note(f"lora infinities, {tokens} tokens")
    c = Case(tokens, tokens, 96, 256, 3, 16)
    c.ids = (np.arange(tokens) % 3).astype(np.int32)
    c.ids[5] = -1
    clean = c.run()
    c.a[1, 3, 7], c.b[1, :, 2], c.scale[2] = 0x7F80, 0x7FC0, np.nan
    y = c.run()
    assert torch.equal(y[c.ids < 1], clean[c.ids < 1])
    assert torch.isnan(y[c.ids == 1]).all() and torch.isnan(y[c.ids == 2]).all()
    # and a token's stay its own
    c = Case(tokens, tokens, 96, 256, 3, 16, 1)
    clean = c.run()
    c.x[4, 9] = 0x7FC0
    y = c.run()
    rest = [t for t in range(tokens) if t != 4]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[4]).all()


def test_strides_and_any_workspace_give_the_same_bits():
    note("lora strides")
    for tokens in (7, 90, 260):
        c = Case(tokens, tokens, 100, 272, 4, 16)
        y = c.run()
        wide = torch.full((tokens, 288), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :272] = to_dev_bf16(c.x)
        out = torch.full((tokens, 107), 5.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.zeros(nq.matmul_lora_workspace_bytes(*c.dims) + 64, dtype=torch.uint8, device=DEV)
        got = c.run(x=wide[:, :272], out=out[:, :100], ws=ws[16:])
        assert torch.equal(got, y) and (out[:, 100:] == 5).all()


def test_adapters_past_four_gigabytes():
    """The last of 700 adapters begins 6 GB on."""
    note("lora adapters past 4 GiB")
    tokens, out, k, rank = 3, 64, 16384, 256
    n = 700
    c = Case(1, tokens, out, k, 1, rank, n - 1)
    a = torch.zeros(n, rank, k, dtype=torch.bfloat16, device=DEV)
    b = torch.zeros(n, out, rank, dtype=torch.bfloat16, device=DEV)
    scale = torch.zeros(n, device=DEV)
    a[-1], b[-1], scale[-1] = to_dev_bf16(c.a[0]), to_dev_bf16(c.b[0]), float(c.scale[0])
    y = nq.matmul_w4a16_lora(to_dev_bf16(c.x), *c.args()[:4], a, b, scale)
    c.ids[:] = 0
    c.check(y)


def test_integers_are_exact():
    """Whole numbers whose sums bf16 holds: every adapter's own columns and rank."""
    note("lora integers")
    for tokens in (16, 48, 300):
        k, out, n, rank = 64, 80, 5, 40
        rng = np.random.default_rng(tokens)
        x = torch.zeros(tokens, k, dtype=torch.bfloat16, device=DEV)
        at = torch.from_numpy(rng.integers(0, k, tokens)).to(DEV)
        x[torch.arange(tokens, device=DEV), at] = 1                        # picks a column of A
        a = torch.zeros(n, rank, k, dtype=torch.bfloat16, device=DEV)
        row = torch.arange(k, device=DEV) * 7 % rank
        a[:, row, torch.arange(k, device=DEV)] = 1                         # whose one is in that row
        b = torch.from_numpy(rng.integers(-100, 101, (n, out, rank))).to(DEV, torch.bfloat16)
        ids = torch.from_numpy(rng.integers(0, n, tokens).astype(np.int32)).to(DEV)
        p = torch.zeros(out, k // 2, dtype=torch.uint8, device=DEV)
        c = torch.zeros(out, k // 16, dtype=torch.uint8, device=DEV)
        y = nq.matmul_w4a16_lora(x, p, c, torch.ones(1, device=DEV), ids, a, b, torch.full((n,), 2.0, device=DEV))
        assert torch.equal(y.float(), 2 * b[ids.long(), :, row[at]].float())
