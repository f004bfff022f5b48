"""The expert layer over sorted tokens against float64.

Bounds: sums of n products in fp32 are off by n 2^-23 of the sum of magnitudes
(whatever the order, tensor scales and weights included); silu * up, made of
fp32 functions good to a few 2^-22, is rounded to bf16, 2^-8 of its value, and so
is y; an expert's row is rounded to fp16, 2^-11 of its value, or, 2^28 and more
below the largest of its 32 columns, to 2^-39 of that one (half of fp16's last step
2^-24 where the largest is 2^14 or more).  That is the worst case; rounding errors
are spread evenly over half a step and independent, so over many outputs the three
of them make a relative error of sqrt((2 + 2^-6) / 3) 2^-8 at most, and y's is held
to 2^-8 of its norm."""
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
    """A layer, its oracle values and inputs."""

    def __init__(self, seed, tokens, hidden, inter, experts, top_k, ids=None):
        rng = np.random.default_rng(seed)
        self.tokens, self.hidden, self.inter, self.experts, self.top_k = tokens, hidden, inter, experts, top_k
        def weights(mats, rows, k):
            p = rng.integers(0, 256, (experts, mats, rows, k // 2), dtype=np.uint8)
            c = rng.integers(0x28, 0x60, (experts, mats, rows, k // 16), dtype=np.uint8)
            c[rng.random(c.shape) < 0.02] = 0
            c[rng.random(c.shape) < 0.02] = 3                # subnormal scales
            s = (2.0 ** -rng.integers(2, 5, experts) / np.sqrt(k) / 3).astype(np.float32)
            return p, c, s
        self.w = [*weights(2, inter, hidden), *weights(1, hidden, inter)]
        self.x = F.f64_to_bf16_bits(rng.standard_normal((tokens, hidden)))
        self.ids = (rng.integers(-1, experts, (tokens, top_k)) if ids is None else ids(rng)).astype(np.int32)
        self.wt = rng.random((tokens, top_k)).astype(np.float32)
        self.dev = [to_dev_f32(a) if a.dtype == np.float32 else to_dev_u8(a) for a in self.w]

    def run(self, x=None, out=None, ws=None):
        x = to_dev_bf16(self.x) if x is None else x
        if ws is None:
            n = nq.moe_sorted_workspace_bytes(self.tokens, self.top_k, self.experts, self.hidden, self.inter)
            ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        return nq.moe_forward_sorted(x, torch.from_numpy(self.ids).to(DEV), to_dev_f32(self.wt), *self.dev, out=out,
                                     workspace=ws)

    def want(self):
        p13, c13, s13, p2, c2, s2 = self.w
        return L.moe_forward_sorted(F.bf16_bits_to_f64(self.x), self.ids, self.wt.astype(np.float64),
                                    O.nvfp4_values(p13, c13, s13), O.nvfp4_values(p2, c2, s2)[:, 0], EPS,
                                    HALF + 32 * EPS, 2.0 ** -11)

    def check(self, y):
        got = F.bf16_bits_to_f64(to_host_bits(y))
        ref, off = self.want()
        bound = HALF * np.abs(ref) + off * (1 + HALF) + 2.0 ** -120
        assert np.all(np.abs(got - ref) <= bound), f"{np.max(np.abs(got - ref) / bound):.3f} of the bound"
        assert np.linalg.norm(got - ref) <= HALF * np.linalg.norm(ref)


# rows an expert: under 32, 64, 128, 256 and beyond; hidden and inter off the stages' 64 and the tiles' rows
SIZES = [(65, 64, 48, 8, 2), (100, 528, 160, 24, 4), (300, 1024, 544, 16, 3), (200, 48, 16, 5, 1), (200, 272, 208, 4, 1),
         (500, 512, 96, 8, 2), (1000, 128, 336, 8, 2), (1500, 256, 272, 4, 2), (700, 640, 528, 2, 1), (65, 16, 16, 1, 1),
         (130, 7168, 64, 16, 2), (130, 80, 2064, 3, 2), (70, 64, 64, 1024, 16)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", SIZES)
def test_layer(tokens, hidden, inter, experts, top_k):
    note(f"layer {tokens}x{top_k} of {experts}, {hidden} -> {inter}")
    c = Case(tokens + hidden, tokens, hidden, inter, experts, top_k)
    c.check(c.run())


@pytest.mark.parametrize("tokens", [1, 17, 64])
def test_few_tokens_are_moe_forward(tokens):
    note(f"layer of {tokens} tokens")
    c = Case(tokens, tokens, 256, 96, 8, 2)
    y = c.run()
    c.check(y)
    assert torch.equal(y, nq.moe_forward(to_dev_bf16(c.x), torch.from_numpy(c.ids).to(DEV), to_dev_f32(c.wt), *c.dev))


IDS = {
    "one expert": lambda t, k, e: lambda r: np.full((t, k), e - 1),
    "the same twice": lambda t, k, e: lambda r: np.repeat(r.integers(0, e, (t, 1)), k, 1),
    "few experts": lambda t, k, e: lambda r: r.choice([0, e // 2], (t, k)),
    "far outside": lambda t, k, e: lambda r: r.choice([-2 ** 31, -1, 0, e - 1, e, 2 ** 31 - 1], (t, k)),
    "skewed": lambda t, k, e: lambda r: np.minimum(r.geometric(0.5, (t, k)) - 1, e - 1),
}


@pytest.mark.parametrize("kind", list(IDS))
@pytest.mark.parametrize("tokens,experts", [(150, 16), (600, 4)])
def test_choices(kind, tokens, experts):
    note(f"layer {kind} {tokens} of {experts}")
    c = Case(tokens, tokens, 192, 144, experts, 3, IDS[kind](tokens, 3, experts))
    c.check(c.run())


def test_no_choice_gives_zeros_and_leaves_what_is_beside():
    note("layer without choices")
    c = Case(1, 90, 64, 32, 4, 2, lambda r: np.full((90, 2), -1))
    out = torch.full((91, 80), 5.0, dtype=torch.bfloat16, device=DEV)
    c.run(out=out[:90, :64])
    assert not out[:90, :64].any() and (out[:90, 64:] == 5).all() and (out[90:] == 5).all()


def test_strided_tokens_and_any_workspace_give_the_same_bits():
    note("layer strided")
    c = Case(2, 333, 272, 80, 8, 4)
    y = c.run()
    wide = torch.full((333, 288), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :272] = to_dev_bf16(c.x)
    n = nq.moe_sorted_workspace_bytes(333, 4, 8, 272, 80)
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device=DEV)
    assert torch.equal(c.run(x=wide[:, :272], ws=ws[256:]), y)
    assert torch.equal(c.run(), y)


def test_more_choices_than_a_pass():
    """144000 choices go in two passes; a token's result does not depend on its pass."""
    note("layer in passes")
    c = Case(3, 9000, 48, 32, 8, 16)
    y = c.run()
    c.check(y)


def test_tokens_past_two_gigabytes():
    """x's rows are 32 MiB apart: 64 of them have 32-bit offsets."""
    note("layer, tokens past 2 GiB")
    c = Case(4, 70, 64, 32, 4, 2)
    big = torch.empty(70, 1 << 24, dtype=torch.bfloat16, device=DEV)
    big[:, :64] = to_dev_bf16(c.x)
    y = c.run(x=big[:, :64])
    c.check(y)


@pytest.mark.parametrize("tokens", [70, 400])
def test_infinite_values_stay_with_their_tokens(tokens):
    note(f"layer, infinite values, {tokens} tokens")
    c = Case(5, tokens, 64, 32, 4, 2, lambda r: r.integers(0, 4, (tokens, 2)))
    clean = c.run()
    c.x[3, 5], c.x[7, 9] = 0x7F80, 0x7FC0
    c.wt[11, 1] = np.inf
    y = c.run()
    same = [t for t in range(tokens) if t not in (3, 7, 11)]
    assert torch.equal(y[same], clean[same])
    assert not torch.isfinite(y[7]).any() and not torch.isfinite(y[11]).all() and not torch.isfinite(y[3]).all()


def test_nan_scale_reaches_its_expert_s_tokens_alone():
    note("layer, NaN scale")
    c = Case(6, 200, 64, 32, 4, 1, lambda r: np.arange(200)[:, None] % 4)
    c.w[1][2, 1, 5, 1] = 0x7F
    c.dev[1] = to_dev_u8(c.w[1])
    y = c.run()
    assert torch.isnan(y[2::4]).all() and torch.isfinite(y[0::4]).all() and torch.isfinite(y[1::4]).all() and \
        torch.isfinite(y[3::4]).all()


def test_large_gates():
    """exp(-gate) overflows and underflows: silu goes to 0 and to gate."""
    note("layer, large gates")
    c = Case(7, 128, 64, 32, 4, 2)
    c.w[2][:] *= 300
    c.dev[2] = to_dev_f32(c.w[2])
    with np.errstate(over="ignore"):
        c.check(c.run())
