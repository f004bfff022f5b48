"""The layer oracle against plain loops, numpy's stable sort, differences and the
expert layer of product.py."""
import numpy as np

import oracle as O
from oracle import layer as L


def _case(seed, tokens=23, top_k=3, experts=5, cols=16):
    rng = np.random.default_rng(seed)
    ids = rng.integers(-2, experts + 2, (tokens, top_k)).astype(np.int32)
    return rng, ids, *L.moe_sort(ids, experts)


def test_sort_is_a_stable_sort():
    _, ids, order, place, offsets = _case(0)
    flat = ids.reshape(-1)
    inside = np.flatnonzero((flat >= 0) & (flat < 5))
    want = inside[np.argsort(flat[inside], kind="stable")]
    n = want.size
    assert offsets[-1] == n and np.array_equal(order[:n], want) and (order[n:] == -1).all()
    assert np.array_equal(place.reshape(-1)[want], np.arange(n)) and (np.delete(place.reshape(-1), inside) == -1).all()
    for e in range(5):
        assert (flat[order[offsets[e]:offsets[e + 1]]] == e).all()


def test_there_and_back():
    rng, ids, order, place, offsets = _case(1)
    x = rng.standard_normal((23, 16))
    xs = L.moe_dispatch(x, place, np.full((69, 16), 7.0))
    n = offsets[-1]
    assert np.array_equal(xs[:n], x[order[:n] // 3]) and (xs[n:] == 7).all()
    y, mag = L.moe_combine(xs, place)
    assert np.allclose(y, x * (place >= 0).sum(1)[:, None]) and np.allclose(mag, np.abs(y))


def test_gradient_by_differences():
    rng, ids, order, place, offsets = _case(2)
    n = offsets[-1]
    ys, w, dy = rng.standard_normal((69, 16)), rng.random((23, 3)), rng.standard_normal((23, 16))
    dys, dw, _ = L.moe_combine_grad(dy, ys, place, w)
    loss = lambda ys, w: (L.moe_combine(ys, place, w)[0] * dy).sum()      # linear in either
    for _ in range(20):
        r, c, t, s = rng.integers(n), rng.integers(16), rng.integers(23), rng.integers(3)
        a, b = ys.copy(), w.copy()
        a[r, c] += 1.0
        b[t, s] += 1.0
        assert np.isclose(loss(a, w) - loss(ys, w), dys[r, c]) and np.isclose(loss(ys, b) - loss(ys, w), dw[t, s])
    assert np.isnan(dys[n:]).all()


def test_layer_is_that_of_product():
    rng, ids, *_ = _case(3)
    x, w13, w2 = rng.standard_normal((23, 16)), rng.standard_normal((5, 2, 8, 16)), rng.standard_normal((5, 16, 8))
    wts = rng.random((23, 3))
    y, off = L.moe_forward_sorted(x, ids, wts, w13, w2, 0.0, 0.0, 0.0)
    assert np.allclose(y, O.moe_forward(x, ids, wts, w13, w2)[0]) and not off.any()
    assert (L.moe_forward_sorted(x, ids, wts, w13, w2, 1e-7, 1e-3, 1e-4)[1] >= 0).all()


def test_lora_is_a_sum_over_tokens():
    rng = np.random.default_rng(4)
    x, w, a, b = (rng.standard_normal(s) for s in ((9, 16), (12, 16), (3, 8, 16), (3, 12, 8)))
    ids, scale = rng.integers(-1, 4, 9), rng.random(3)
    y, _ = L.matmul_lora(x, w, ids, a, b, scale, 0.0)
    for t in range(9):
        m = w + (scale[ids[t]] * b[ids[t]] @ a[ids[t]] if 0 <= ids[t] < 3 else 0.0)
        assert np.allclose(y[t], m @ x[t])
