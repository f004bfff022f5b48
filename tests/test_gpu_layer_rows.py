"""Tokens sorted by expert and back, and the gradient, against float64.

Sums of n fused products in fp32 are off by at most n 2^-24 of the sum of
magnitudes, whatever their order; a bf16 result by half a step more, 2^-8 of its
value (2^-134 below the smallest normal one)."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq
from oracle import formats as F
from oracle import layer as L

from _gpu import DEV, host, need_gpu, note, to_dev_bf16, to_dev_f32, to_host_bits

pytestmark = pytest.mark.gpu

HALF, EPS = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _ids(rng, tokens, top_k, experts, kind):
    if kind == "none":
        return np.full((tokens, top_k), -1, np.int32)
    if kind == "one":
        return np.full((tokens, top_k), experts - 1, np.int32)
    if kind == "mixed":                                  # some elsewhere, the same one twice
        return rng.integers(-2, experts + 3, (tokens, top_k)).astype(np.int32)
    ids = rng.integers(0, experts, (tokens, top_k)).astype(np.int32)
    if kind == "extreme":
        ids[rng.random(ids.shape) < 0.3] = 2 ** 31 - 1
        ids[rng.random(ids.shape) < 0.3] = -2 ** 31
    return ids


def _bits(rng, *shape):
    return F.f64_to_bf16_bits(rng.standard_normal(shape))


def _vals(t):
    return F.bf16_bits_to_f64(to_host_bits(t))


def _rounded(got, ref, mag, n):
    bound = HALF * np.abs(ref) + n * EPS * mag * (1 + HALF) + 2.0 ** -134
    assert np.all(np.abs(got - ref) <= bound)


# one workgroup and several, experts off powers of two, one choice, the most places
SORTS = [(1, 1, 1), (1, 16, 1024), (61, 8, 128), (63, 1, 3), (1024, 8, 128), (1025, 8, 129), (4097, 3, 24), (70000, 8, 128),
         (9001, 16, 1024), (300001, 1, 7)]


@pytest.mark.parametrize("kind", ["spread", "mixed", "one", "none", "extreme"])
@pytest.mark.parametrize("tokens,top_k,experts", SORTS)
def test_sort(tokens, top_k, experts, kind):
    note(f"sort {tokens}x{top_k} of {experts} {kind}")
    ids = _ids(np.random.default_rng(tokens + experts), tokens, top_k, experts, kind)
    flat = ids.reshape(-1)
    inside = np.flatnonzero((flat >= 0) & (flat < experts))
    want = inside[np.argsort(flat[inside], kind="stable")]
    dev = torch.from_numpy(ids).to(DEV)
    ws = torch.full((max(nq.moe_sort_workspace_bytes(tokens, top_k, experts), 1),), 255, dtype=torch.uint8, device=DEV)
    order, place, offsets = (host(t) for t in nq.moe_sort(dev, experts, workspace=ws))
    n = want.size
    assert np.array_equal(order[:n], want) and (order[n:] == -1).all()
    back = np.full(flat.size, -1)
    back[want] = np.arange(n)
    assert np.array_equal(place.reshape(-1), back)
    assert np.array_equal(offsets, np.searchsorted(flat[want], np.arange(experts + 1)))


def test_sort_of_no_tokens():
    note("sort of no tokens")
    order, place, offsets = nq.moe_sort(torch.empty(0, 4, dtype=torch.int32, device=DEV), 9)
    assert order.numel() == 0 and place.shape == (0, 4) and not host(offsets).any()


@pytest.mark.parametrize("tokens,top_k,cols,dtype", [
    (1, 1, 8, torch.bfloat16), (61, 8, 7168, torch.bfloat16), (300, 3, 2056, torch.bfloat16), (77, 16, 33, torch.uint8),
    (77, 2, 3, torch.uint8), (50, 4, 12, torch.uint8), (129, 5, 100, torch.float32), (9, 2, 5, torch.bfloat16),
    (1000, 1, 16, torch.uint8)])
def test_dispatch(tokens, top_k, cols, dtype):
    note(f"dispatch {tokens}x{top_k} cols={cols} {dtype}")
    rng = np.random.default_rng(tokens)
    ids = _ids(rng, tokens, top_k, 6, "mixed")
    _, place, offsets = nq.moe_sort(torch.from_numpy(ids).to(DEV), 6)
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    size = torch.empty(0, dtype=dtype).element_size()
    x = torch.randint(0, 256, (tokens, cols * size), generator=g, device=DEV, dtype=torch.uint8).view(dtype)
    old = torch.full((tokens * top_k, cols * size), 0x5A, device=DEV, dtype=torch.uint8).view(dtype)
    got = nq.moe_dispatch(x, place, out=old.clone())
    want = L.moe_dispatch(host(x.view(torch.uint8)), host(place), host(old.view(torch.uint8)))
    assert np.array_equal(host(got.view(torch.uint8)), want)
    # strided rows, both sides
    wide_x = torch.zeros(tokens, cols + 16 // size * 3, device=DEV, dtype=dtype)
    wide_o = torch.zeros(tokens * top_k, cols + 16 // size, device=DEV, dtype=dtype)
    wide_x[:, :cols], wide_o[:, :cols] = x, old
    got = nq.moe_dispatch(wide_x[:, :cols], place, out=wide_o[:, :cols])
    assert np.array_equal(host(got.contiguous().view(torch.uint8)), want) and not wide_o[:, cols:].any()


ROWS = [(1, 1, 8), (61, 8, 7168), (300, 3, 2056), (77, 16, 520), (129, 5, 512), (1000, 2, 16), (40, 4, 1048)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,top_k,cols", ROWS)
def test_combine(tokens, top_k, cols, weighted):
    note(f"combine {tokens}x{top_k} cols={cols} weighted={weighted}")
    rng = np.random.default_rng(tokens + cols)
    ids = _ids(rng, tokens, top_k, 6, "mixed")
    ids[0] = -1                                          # a token without an expert
    place = L.moe_sort(ids, 6)[1]
    ys, w = _bits(rng, tokens * top_k, cols), rng.standard_normal((tokens, top_k)).astype(np.float32)
    ys[(place >= 0).sum():] = 0x7FC0                     # rows behind the last hold NaN
    w[place < 0] = np.nan
    y = nq.moe_combine(to_dev_bf16(ys), torch.from_numpy(place).to(DEV), to_dev_f32(w) if weighted else None)
    ref, mag = L.moe_combine(F.bf16_bits_to_f64(ys), place, w.astype(np.float64) if weighted else None)
    _rounded(_vals(y), ref, mag, top_k)
    assert not _vals(y)[0].any()


@pytest.mark.parametrize("tokens,top_k,cols", ROWS)
def test_combine_grad(tokens, top_k, cols):
    note(f"combine_grad {tokens}x{top_k} cols={cols}")
    rng = np.random.default_rng(tokens + cols + 1)
    ids = _ids(rng, tokens, top_k, 6, "mixed")
    place = L.moe_sort(ids, 6)[1]
    n = int((place >= 0).sum())
    dy, ys = _bits(rng, tokens, cols), _bits(rng, tokens * top_k, cols)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    ys[n:] = 0x7FC0
    w[place < 0] = np.nan
    old = torch.full((tokens * top_k, cols), 3.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((tokens, top_k), np.nan, device=DEV)
    got, gw = nq.moe_combine_grad(to_dev_bf16(dy), to_dev_bf16(ys), torch.from_numpy(place).to(DEV), to_dev_f32(w),
                                  out=(old, dw))
    assert got is old and gw is dw
    dys, rw, mag = L.moe_combine_grad(F.bf16_bits_to_f64(dy), F.bf16_bits_to_f64(ys), place, w.astype(np.float64))
    _rounded(_vals(got)[:n], dys[:n], np.abs(dys[:n]), 1)
    assert (_vals(got)[n:] == 3).all()
    assert np.all(np.abs(host(gw) - rw) <= cols * EPS * mag * 1.001)
    # dispatch's gradient is the sum of the rows
    dx = nq.moe_dispatch_grad(got, torch.from_numpy(place).to(DEV))
    ref, mag = L.moe_combine(_vals(got), place)
    _rounded(_vals(dx), ref, mag, top_k)


def test_gradient_by_differences():
    """combine is linear in ys and in the weights: differences of its float32
    result, made of many bf16 ones, agree with the gradient."""
    note("gradient by differences")
    rng = np.random.default_rng(5)
    place = torch.from_numpy(L.moe_sort(_ids(rng, 6, 3, 4, "mixed"), 4)[1]).to(DEV)
    # small whole numbers: every sum is exact in bf16
    ys = torch.from_numpy(rng.integers(-3, 4, (18, 32))).to(DEV, torch.bfloat16)
    dy = torch.from_numpy(rng.integers(-2, 3, (6, 32))).to(DEV, torch.bfloat16)
    w = torch.from_numpy(rng.integers(1, 4, (6, 3))).to(DEV, torch.float32)
    loss = lambda ys, w: float((nq.moe_combine(ys, place, w).double() * dy.double()).sum())
    base = loss(ys, w)
    dys, dw = nq.moe_combine_grad(dy, ys, place, w)
    for t in range(6):
        for s in range(3):
            v = w.clone()
            v[t, s] += 1
            assert loss(ys, v) - base == float(dw[t, s])
            r = int(place[t, s])
            if r >= 0:
                v = ys.clone()
                v[r, 7] += 1
                assert loss(v, w) - base == float(dys[r, 7])


def test_strided_rows_and_places_outside():
    """Rows 16 bytes and more apart; places beyond the rows add and get nothing."""
    note("strided rows, places outside")
    rng = np.random.default_rng(9)
    tokens, top_k, cols = 37, 4, 136
    ids = _ids(rng, tokens, top_k, 6, "spread")
    place = L.moe_sort(ids, 6)[1]
    bad = place.copy()
    bad[::3, 1] = tokens * top_k
    bad[1::3, 2] = -7
    bad[2::3, 0] = 2 ** 31 - 1
    clean = np.where((bad >= 0) & (bad < tokens * top_k), bad, -1)
    ysb, dyb = _bits(rng, tokens * top_k, cols), _bits(rng, tokens, cols)
    ys = torch.zeros(tokens * top_k, cols + 24, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros(tokens, cols + 8, dtype=torch.bfloat16, device=DEV)
    out = torch.full((tokens, cols + 40), 5.0, dtype=torch.bfloat16, device=DEV)
    ys[:, :cols], dy[:, :cols] = to_dev_bf16(ysb), to_dev_bf16(dyb)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    p = torch.from_numpy(bad).to(DEV)
    y = nq.moe_combine(ys[:, :cols], p, to_dev_f32(w), out=out[:, :cols])
    ref, mag = L.moe_combine(F.bf16_bits_to_f64(ysb), clean, w.astype(np.float64))
    _rounded(_vals(y), ref, mag, top_k)
    assert (out[:, cols:] == 5).all()
    dys = torch.full((tokens * top_k, cols + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    got, gw = nq.moe_combine_grad(dy[:, :cols], ys[:, :cols], p, to_dev_f32(w),
                                  out=(dys[:, :cols], torch.empty(tokens, top_k, device=DEV)))
    rd, rw, mag = L.moe_combine_grad(F.bf16_bits_to_f64(dyb), F.bf16_bits_to_f64(ysb), clean, w.astype(np.float64))
    hit = ~np.isnan(rd[:, 0])
    _rounded(_vals(got)[hit], rd[hit], np.abs(rd[hit]), 1)
    assert (_vals(got)[~hit] == 5).all() and (dys[:, cols:] == 5).all()
    assert np.all(np.abs(host(gw) - rw) <= cols * EPS * mag * 1.001) and not host(gw)[clean < 0].any()


def test_infinities_and_nan_stay_with_their_token():
    note("infinities stay with their token")
    place = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    ys = torch.ones(8, 16, dtype=torch.bfloat16, device=DEV)
    ys[2], ys[5, 3] = float("inf"), float("nan")
    w = torch.ones(4, 2, device=DEV)
    y = nq.moe_combine(ys, place, w)
    assert (y[[0, 3]] == 2).all() and torch.isinf(y[1]).all() and torch.isnan(y[2, 3]) and (y[2, :3] == 2).all()
    w[0, 0] = float("nan")
    assert torch.isnan(nq.moe_combine(ys, place, w)[0]).all()
    dys, dw = nq.moe_combine_grad(torch.ones(4, 16, dtype=torch.bfloat16, device=DEV), ys, place, w)
    assert torch.isnan(dys[0]).all() and (dys[1:] == 1).all()
    assert torch.isinf(dw[1, 0]) and torch.isnan(dw[2, 1]) and dw[0, 0] == 16 and dw[3, 1] == 16


def test_rows_past_four_gigabytes():
    """8 GiB of sorted rows: the last ones lie beyond 32-bit offsets."""
    note("rows past 4 GiB")
    tokens, top_k, cols = 65536, 8, 8192
    place = torch.arange(tokens * top_k, dtype=torch.int32, device=DEV).flip(0).view(tokens, top_k).contiguous()
    x = (torch.arange(tokens, device=DEV) % 251).to(torch.bfloat16)[:, None].expand(tokens, cols).contiguous()
    xs = nq.moe_dispatch(x, place)
    want = (torch.arange(tokens * top_k, device=DEV).flip(0) // top_k % 251).to(torch.bfloat16)
    assert torch.equal(xs[:, 0], want) and torch.equal(xs[:, -1], want)
    assert torch.equal(nq.moe_combine(xs, place, torch.full((tokens, top_k), 0.125, device=DEV)), x)
    ones = torch.ones(tokens, top_k, device=DEV)
    dys, dw = nq.moe_combine_grad(x, xs, place, ones)
    assert torch.equal(dys[:, 0], want) and torch.equal(dys[:, -1], want)
    v = (torch.arange(tokens, device=DEV) % 251).double() ** 2 * cols
    assert torch.allclose(dw.double(), v[:, None].expand(-1, top_k), rtol=cols * EPS, atol=0)
