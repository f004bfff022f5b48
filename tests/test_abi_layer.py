"""C ABI of the layer library without a GPU: its header, exports and binding are
one list, and bad arguments are refused before any HIP call.

Pointers used here are never dereferenced: every call is built to fail
validation, or to have nothing to do."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import nvfp4_post_quantization_amd as nq
from nvfp4_post_quantization_amd import layer

OK, NULL, SHAPE, ALIGN, WS, BADIN = 0, 1, 2, 3, 4, 5
P = 0x10000
HEADER = os.path.join(os.path.dirname(layer.__file__), "include", "nvfp4mi_layer.h")
ABI = {
    "nvfp4_moe_sort_workspace_bytes", "nvfp4_moe_sort", "nvfp4_moe_dispatch", "nvfp4_moe_combine",
    "nvfp4_moe_combine_grad", "nvfp4_moe_forward_sorted_workspace_bytes", "nvfp4_moe_forward_sorted",
    "nvfp4_matmul_w4a16_lora_workspace_bytes", "nvfp4_matmul_w4a16_lora",
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(layer.LIB_PATH):
        pytest.skip("libnvfp4mi_layer.so not built")
    return layer.load()


def test_header_exports_and_binding_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    text = re.sub(r"^\s*#.*$", "", text, flags=re.M)
    assert set(re.findall(r"(\w+)\s*\([^(){};]*\)\s*;", text)) == ABI == set(layer._SIGS)
    if not shutil.which("nm"):
        pytest.skip("no nm")
    out = subprocess.run(["nm", "-D", "--defined-only", layer.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert {l.split()[2] for l in out.splitlines() if l.split()[1] == "T" and not l.split()[2].startswith("_")} == ABI


def test_functions_are_the_package_s():
    for n in layer.__all__:
        assert getattr(nq, n) is getattr(layer, n) and n in nq.__all__


def test_header_compiles_as_c():
    if not shutil.which("gcc"):
        pytest.skip("no gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-x", "c", "-I",
                    os.path.join(root, "include"), HEADER], check=True)


def test_sort_validation(lib):
    f, need = lib.nvfp4_moe_sort, lib.nvfp4_moe_sort_workspace_bytes
    call = lambda ids=P, t=4, k=2, e=8, o=P, p=P, off=P, ws=P, n=1 << 30: f(ids, t, k, e, o, p, off, ws, n, None)
    for k in (0, -1, 17):
        assert call(k=k) == BADIN and need(4, k, 8) == 0
    for e in (0, -1, 1025):
        assert call(e=e) == BADIN and need(4, 2, e) == 0
    assert call(t=-1) == SHAPE and call(t=(1 << 29) + 1) == SHAPE and need((1 << 29) + 1, 2, 8) == 0
    assert call(t=(1 << 29), ws=P + 2) == ALIGN
    for a in ("ids", "o", "p", "off"):
        assert call(**{a: None}) == NULL
        assert call(**{a: P + 2}) == ALIGN
    n = need(100000, 8, 128)
    assert n > 0 and call(t=100000, k=8, e=128, n=n - 1) == WS and call(t=100000, k=8, e=128, n=n, ws=None) == NULL
    assert need(61, 8, 128) == 0 and need(0, 8, 128) == 0


def test_dispatch_validation(lib):
    f = lib.nvfp4_moe_dispatch
    call = lambda x=P, t=4, b=32, ld=32, p=P, k=2, xs=P, ldxs=32: f(x, t, b, ld, p, k, xs, ldxs, None)
    assert call(k=0) == BADIN and call(k=17) == BADIN
    assert call(t=-1) == SHAPE and call(b=0) == SHAPE and call(ld=31) == SHAPE and call(ldxs=31) == SHAPE
    assert call(t=1 << 28, ldxs=1 << 40) == SHAPE
    for a in ("x", "p", "xs"):
        assert call(**{a: None}) == NULL
    assert call(p=P + 1) == ALIGN
    assert call(x=None, p=None, xs=None, t=0) == OK


def test_combine_validation(lib):
    f = lib.nvfp4_moe_combine
    call = lambda ys=P, ld=32, p=P, w=P, t=4, k=2, c=32, y=P, ldy=32: f(ys, ld, p, w, t, k, c, y, ldy, None)
    assert call(k=0) == BADIN and call(k=17) == BADIN
    assert call(c=12) == SHAPE and call(c=0) == SHAPE and call(ld=24) == SHAPE and call(ldy=24) == SHAPE and call(t=-2) == SHAPE
    for a in ("ys", "p", "y"):
        assert call(**{a: None}) == NULL
    for a in ("ys", "y"):
        assert call(**{a: P + 8}) == ALIGN
    for a in ("ld", "ldy"):
        assert call(**{a: 36}) == ALIGN
    assert call(p=P + 2) == ALIGN and call(w=P + 2) == ALIGN
    assert call(ys=None, p=None, w=None, y=None, t=0) == OK


def test_combine_grad_validation(lib):
    f = lib.nvfp4_moe_combine_grad
    call = lambda dy=P, lddy=32, ys=P, ldys=32, p=P, w=P, t=4, k=2, c=32, dys=P, lddys=32, dw=P: f(
        dy, lddy, ys, ldys, p, w, t, k, c, dys, lddys, dw, None)
    assert call(k=0) == BADIN and call(k=17) == BADIN
    assert call(c=4) == SHAPE and call(t=-2) == SHAPE
    for a in ("lddy", "ldys", "lddys"):
        assert call(**{a: 24}) == SHAPE and call(**{a: 36}) == ALIGN
    for a in ("dy", "ys", "p", "w", "dys", "dw"):
        assert call(**{a: None}) == NULL
    for a in ("dy", "ys", "dys"):
        assert call(**{a: P + 8}) == ALIGN
    for a in ("p", "w", "dw"):
        assert call(**{a: P + 2}) == ALIGN
    assert call(t=0, dy=None, ys=None, p=None, w=None, dys=None, dw=None) == OK


def test_layer_validation(lib):
    f, need = lib.nvfp4_moe_forward_sorted, lib.nvfp4_moe_forward_sorted_workspace_bytes
    names = ["x", "t", "d", "ldx", "ids", "w", "k", "e", "f", "p13", "c13", "s13", "p2", "c2", "s2", "y", "ldy", "ws", "n"]
    base = dict(x=P, t=100, d=64, ldx=64, ids=P, w=P, k=2, e=8, f=32, p13=P, c13=P, s13=P, p2=P, c2=P, s2=P, y=P, ldy=64,
                ws=P, n=1 << 40)
    call = lambda **kw: f(*[{**base, **kw}[a] for a in names], None)
    assert call(k=0) == BADIN and call(k=17) == BADIN and call(e=0) == BADIN and call(e=1025) == BADIN
    for kw in (dict(t=-1), dict(t=(1 << 29) + 1), dict(d=24), dict(d=0), dict(f=24), dict(f=0), dict(ldx=48), dict(ldy=48),
               dict(d=(1 << 17) + 16, ldx=1 << 18, ldy=1 << 18), dict(f=(1 << 17) + 16),
               dict(d=1 << 17, f=1 << 14, ldx=1 << 18, ldy=1 << 18)):
        assert call(**kw) == SHAPE
    for a in ("x", "ids", "w", "p13", "c13", "s13", "p2", "c2", "s2", "y"):
        assert call(**{a: None}) == NULL
        assert call(**{a: P + 2}) == ALIGN
    assert call(ldx=68) == ALIGN and call(ldy=68) == ALIGN and call(ws=P + 128) == ALIGN
    for t in (1, 64, 65, 100000):
        n = need(t, 2, 8, 64, 32)
        assert n > 0 and call(t=t, n=n - 1) == WS and call(t=t, ws=None, n=n) == NULL
    assert need(0, 2, 8, 64, 32) == 0 and call(t=0, x=None, ids=None, w=None, y=None, ws=None, n=0) == OK
    # more choices than one pass: the workspace stays
    assert need(1 << 20, 8, 8, 64, 32) == need(1 << 17, 8, 8, 64, 32)


def test_lora_validation(lib):
    f, need = lib.nvfp4_matmul_w4a16_lora, lib.nvfp4_matmul_w4a16_lora_workspace_bytes
    names = ["x", "t", "k", "ldx", "p", "c", "s2", "o", "ids", "na", "r", "a", "b", "sc", "y", "ldy", "ws", "n"]
    base = dict(x=P, t=4, k=64, ldx=64, p=P, c=P, s2=P, o=48, ids=P, na=3, r=16, a=P, b=P, sc=P, y=P, ldy=48, ws=P, n=1 << 40)
    call = lambda **kw: f(*[{**base, **kw}[a] for a in names], None)
    for r in (0, 4, 12, 264, -8):
        assert call(r=r) == BADIN and need(4, 48, 64, r) == 0
    assert call(na=-1) == BADIN and call(na=1 << 31) == BADIN
    for kw in (dict(t=-1), dict(t=(1 << 31) - 255), dict(k=24), dict(k=0), dict(o=0, ldy=48), dict(ldx=48), dict(ldy=40)):
        assert call(**kw) == SHAPE
    for a in ("x", "p", "c", "s2", "ids", "a", "b", "sc", "y"):
        assert call(**{a: None}) == NULL
        assert call(**{a: P + 1}) == ALIGN
    assert call(ldx=68) == ALIGN and call(ws=P + 8) == ALIGN
    n = need(4, 48, 64, 16)
    assert n > 0 and call(n=n - 1) == WS and call(ws=None, n=n) == NULL
    assert call(t=0, x=None, ids=None, y=None, ws=None, n=0) == OK


def test_binding_refuses_before_any_call():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    place = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: nq.moe_sort(place, 8), lambda: nq.moe_dispatch(x, place), lambda: nq.moe_combine(x, place),
                 lambda: nq.moe_combine_grad(x, x, place, place.float()),
                 lambda: nq.moe_forward_sorted(x, place, place.float(), x, x, x, x, x, x),
                 lambda: nq.matmul_w4a16_lora(x, x, x, x, place, x, x, x)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(TypeError):
        nq.moe_sort([[1]], 8)
