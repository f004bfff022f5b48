"""C ABI of the packed products without a GPU: the declarations of the header
are exported and bound, and bad arguments are refused before any HIP call.

Pointers used here are never dereferenced: every call is built to fail
validation, or to have nothing to do."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import nvfp4_post_quantization_amd as nq
from nvfp4_post_quantization_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, WS, BADIN = 0, 1, 2, 3, 4, 5
P = 0x10000
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nq.LIB_PATH):
        pytest.skip("libnvfp4mi.so not built")
    return nq.load()


def test_checked_declarations_are_exported_and_bound(lib):
    text = open(os.path.join(ROOT, "include", "nvfp4mi.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^NVFP4_CHECKED\s+\w+\s+(\w+)\s*\(", text, flags=re.M))
    assert names == {"mxfp4_quantize", "mxfp4_dequant", "mxfp4_matmul_workspace_bytes", "mxfp4_matmul",
                     "nvfp4_matmul_workspace_bytes", "nvfp4_matmul_w4a16", "nvfp4_matmul_w4a4", "nvfp4_moe_route",
                     "nvfp4_moe_workspace_bytes", "nvfp4_moe_forward"}
    raw = ctypes.CDLL(nq.LIB_PATH)
    for n in names:
        getattr(raw, n)
        assert n in nq._SIGS


def test_quantize_validation(lib):
    q = lib.mxfp4_quantize
    assert q(P, 4, 48, 48, P, P, None) == SHAPE              # k % 32
    assert q(P, 4, 64, 32, P, P, None) == SHAPE              # ld < k
    assert q(P, -1, 64, 64, P, P, None) == SHAPE
    assert q(P, 1 << 62, 64, 1 << 40, P, P, None) == SHAPE
    assert q(None, 4, 64, 64, P, P, None) == NULL
    assert q(P, 4, 64, 64, None, P, None) == NULL
    assert q(P, 4, 64, 64, P, None, None) == NULL
    assert q(P + 2, 4, 64, 64, P, P, None) == ALIGN
    assert q(P, 4, 64, 68, P, P, None) == ALIGN
    assert q(P, 4, 64, 64, P + 8, P, None) == ALIGN
    assert q(P, 4, 64, 64, P, P + 1, None) == ALIGN
    assert q(None, 0, 64, 64, None, None, None) == OK
    d = lib.mxfp4_dequant
    assert d(P, P, 4, 16, P, None) == SHAPE
    assert d(None, P, 4, 32, P, None) == NULL
    assert d(P, P, 4, 32, P + 2, None) == ALIGN
    assert d(P, P + 1, 4, 32, P, None) == ALIGN
    assert d(None, None, 0, 32, None, None) == OK


def test_mxfp4_matmul_validation(lib):
    f = lib.mxfp4_matmul
    ok = dict(xp=P, xe=P, t=4, k=64, wp=P, we=P, o=5, y=P, ld=5, ws=P, n=1 << 40)
    def call(**kw):
        a = {**ok, **kw}
        return f(a["xp"], a["xe"], a["t"], a["k"], a["wp"], a["we"], a["o"], a["y"], a["ld"], a["ws"], a["n"], None)
    for bad in (dict(k=48), dict(t=-1), dict(o=0), dict(k=0), dict(ld=4), dict(t=BIG), dict(o=BIG, ld=BIG),
                dict(k=BIG), dict(t=1 << 30, ld=1 << 40)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(xp=None), dict(xe=None), dict(wp=None), dict(we=None), dict(y=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(xp=P + 8), dict(xe=P + 4), dict(wp=P + 8), dict(we=P + 1), dict(y=P + 1)):
        assert call(**bad) == ALIGN, bad
    assert call(t=0, xp=None, xe=None, y=None, ws=None, n=0) == OK
    assert call(t=0, wp=None) == NULL


def test_nvfp4_matmul_validation(lib):
    f, g = lib.nvfp4_matmul_w4a16, lib.nvfp4_matmul_w4a4
    ok = dict(x=P, xc=P, xs=P, t=4, k=48, ldx=48, wp=P, wc=P, s=P, o=5, y=P, ld=5, ws=P, n=1 << 40)
    def a16(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["t"], a["k"], a["ldx"], a["wp"], a["wc"], a["s"], a["o"], a["y"], a["ld"], a["ws"], a["n"],
                 None)
    def a4(**kw):
        a = {**ok, **kw}
        return g(a["x"], a["xc"], a["xs"], a["t"], a["k"], a["wp"], a["wc"], a["s"], a["o"], a["y"], a["ld"], a["ws"],
                 a["n"], None)
    for call in (a16, a4):
        for bad in (dict(k=40), dict(t=-1), dict(o=0), dict(ld=4), dict(t=BIG), dict(o=BIG, ld=BIG),
                    dict(k=BIG, ldx=BIG)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(x=None), dict(wp=None), dict(wc=None), dict(s=None), dict(y=None)):
            assert call(**bad) == NULL, bad
        for bad in (dict(x=P + 2), dict(wp=P + 8), dict(wc=P + 2), dict(s=P + 2), dict(y=P + 1)):
            assert call(**bad) == ALIGN, bad
        assert call(t=0, x=None, xc=None, y=None, ws=None, n=0) == OK
        assert call(t=0, s=None) == NULL
    assert a16(ldx=40) == SHAPE and a16(ldx=52) == ALIGN
    assert a4(xc=None) == NULL and a4(xs=None) == NULL and a4(xc=P + 1) == ALIGN and a4(xs=P + 1) == ALIGN


def test_product_workspace(lib):
    for q, unit in ((lib.mxfp4_matmul_workspace_bytes, 32), (lib.nvfp4_matmul_workspace_bytes, 16)):
        for t, o, k in ((-1, 16, 64), (0, 16, 64), (4, 0, 64), (4, 16, unit // 2), (4, 16, 0), (BIG, 16, 64)):
            assert q(t, o, k) == 0
    # a call is refused wherever less than the query's size is given
    for t in (1, 65, 333, 1000, 4095):
        n = lib.mxfp4_matmul_workspace_bytes(t, 4096, 4096)
        if n:
            a = (P, P, t, 4096, P, P, 4096, P, 4096)
            assert lib.mxfp4_matmul(*a, P, n - 1, None) == WS and lib.mxfp4_matmul(*a, None, n, None) == NULL
            assert lib.mxfp4_matmul(*a, P + 8, n, None) == ALIGN
        n = lib.nvfp4_matmul_workspace_bytes(t, 4096, 4096)
        if n:
            a = (P, P, P, t, 4096, P, P, P, 4096, P, 4096)
            assert lib.nvfp4_matmul_w4a4(*a, P, n - 1, None) == WS
            assert lib.nvfp4_matmul_w4a4(*a, None, n, None) == NULL
            assert lib.nvfp4_matmul_w4a4(*a, P + 8, n, None) == ALIGN
            a = (P, t, 4096, 4096, P, P, P, 4096, P, 4096)
            assert lib.nvfp4_matmul_w4a16(*a, P, n - 1, None) == WS


def test_route_validation(lib):
    f = lib.nvfp4_moe_route
    assert f(P, -1, 8, 8, 2, 1, P, P, None) == SHAPE
    assert f(P, 4, 0, 8, 2, 1, P, P, None) == SHAPE
    assert f(P, 4, 8, 7, 2, 1, P, P, None) == SHAPE
    assert f(P, BIG, 8, 8, 2, 1, P, P, None) == SHAPE
    for e, k, n in ((1025, 2, 1), (8, 0, 1), (8, 9, 1), (64, 17, 1), (8, 2, 2), (8, 2, -1)):
        assert f(P, 4, e, e, k, n, P, P, None) == BADIN
    assert f(None, 4, 8, 8, 2, 1, P, P, None) == NULL
    assert f(P, 4, 8, 8, 2, 1, None, P, None) == NULL
    assert f(P, 4, 8, 8, 2, 1, P, None, None) == NULL
    assert f(P + 2, 4, 8, 8, 2, 1, P, P, None) == ALIGN
    assert f(P, 4, 8, 8, 2, 1, P + 1, P, None) == ALIGN
    assert f(None, 0, 8, 8, 2, 1, None, None, None) == OK


def test_moe_validation(lib):
    f, q = lib.nvfp4_moe_forward, lib.nvfp4_moe_workspace_bytes
    assert q(0, 2, 32) == 0 and q(65, 2, 32) == 0 and q(4, 0, 32) == 0 and q(4, 17, 32) == 0 and q(4, 2, 24) == 0
    need = q(4, 2, 32)
    assert need >= 4 * 2 * 32 * 4
    names = "x t hidden ldx ids wt top_k experts inter p13 c13 s13 p2 c2 s2 y ldy ws n".split()
    ok = dict(zip(names, (P, 4, 48, 48, P, P, 2, 8, 32, P, P, P, P, P, P, P, 48, P, need)))
    def call(**kw):
        a = {**ok, **kw}
        return f(*[a[n] for n in names], None)
    for bad in (dict(t=-1), dict(hidden=40), dict(hidden=0), dict(inter=24), dict(inter=0), dict(ldx=40), dict(ldy=40),
                dict(inter=BIG), dict(hidden=BIG, ldx=BIG, ldy=BIG)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(t=65), dict(top_k=0), dict(top_k=17), dict(experts=0), dict(experts=1025)):
        assert call(**bad) == BADIN, bad
    for n in ("x", "ids", "wt", "p13", "c13", "s13", "p2", "c2", "s2", "y", "ws"):
        assert call(**{n: None}) == NULL, n
    for n, off in (("x", 2), ("ids", 2), ("wt", 1), ("p13", 8), ("c13", 2), ("s13", 2), ("p2", 8), ("c2", 8), ("s2", 1),
                   ("y", 1), ("ws", 8)):
        assert call(**{n: P + off}) == ALIGN, n
    assert call(ldx=52) == ALIGN
    assert call(n=need - 1) == WS
    assert call(t=0, x=None, ids=None, wt=None, y=None, ws=None, n=0) == OK
    assert call(t=0, p2=None) == NULL


def test_python_layer_rejects_before_the_library():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    f1 = torch.zeros(1)
    for call in (lambda: nq.mxfp4_quantize(bf(4, 32)), lambda: nq.mxfp4_dequant(u8(4, 16), u8(4, 1)),
                 lambda: nq.mxfp4_matmul(u8(4, 16), u8(4, 1), u8(8, 16), u8(8, 1)),
                 lambda: nq.matmul_w4a16(bf(4, 32), u8(8, 16), u8(8, 2), f1),
                 lambda: nq.matmul_w4a4(u8(4, 16), u8(4, 2), f1, u8(8, 16), u8(8, 2), f1),
                 lambda: nq.moe_route(torch.zeros(4, 8), 2),
                 lambda: nq.moe_forward(bf(4, 32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2),
                                        u8(8, 2, 32, 16), u8(8, 2, 32, 2), torch.zeros(8), u8(8, 32, 16), u8(8, 32, 2),
                                        torch.zeros(8))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        nq.mxfp4_quantize(torch.zeros(4, 32).numpy())


def test_validation_under_sanitizers():
    """The checks above against the build whose argument checks carry
    AddressSanitizer and UndefinedBehaviorSanitizer on their host code."""
    if os.environ.get("NVFP4MI_LIB"):
        return                                              # this is that run
    try:
        rt = B.asan_runtime()
    except Exception as e:                                  # no hipcc / clang runtime in this image
        pytest.skip(f"sanitizer toolchain unavailable: {e}")
    if not os.path.exists(os.path.join(B.BUILD, "moe.o")):
        B.build()
    env = dict(os.environ, LD_PRELOAD=rt, NVFP4MI_LIB=B.build_sanitized(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_abi_product.py", "-q", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
