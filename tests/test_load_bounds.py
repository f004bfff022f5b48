"""Where the expert layer's tiles load, without a GPU.

A buffer load is checked by its lane's offset against the buffer's size less the
scalar offset, as unsigned numbers: with a scalar offset above the size the
difference wraps, and a lane that is meant to read zero (its offset is 2^31) reads
memory 2 GiB on.  Here the loads of one tile are walked through as run_tile issues
them, with the scalar offsets that its source states."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_post_quantization_amd", "csrc",
                      "moe_sorted.hip")
BEYOND = 1 << 31


def _last_argument(call):
    """That of the call that `call` begins with."""
    depth, start = 0, 0
    for i, c in enumerate(call):
        depth += (c in "([{") - (c in ")]}")
        if depth == 1 and c in "(,":
            start = i + 1
        if depth == 0 and c == ")":
            return call[start:i].strip()
    raise ValueError(call)


def _offset(name):
    """The scalar offset that lambda `name` of run_tile gives its loads, as a function."""
    text = re.sub(r"//.*", "", open(SOURCE, encoding="utf-8").read())
    body = re.search(r"const auto %s = \[&\].*?\n  \};" % name, text, re.S).group(0)
    last = _last_argument(re.sub(r"<[^;(]*?>(?=\()", "", body[body.index("load_lds"):]))
    given = re.search(r"const int %s = ([^;]*);" % re.escape(last), body)
    code = compile((given.group(1) if given else last).replace("(int)", "").strip(), name, "eval")
    return lambda **v: eval(code, {"min": min, **v})  # noqa: S307  (an expression of this repository)


def _stages(k, tm):
    """(stages of x, pairs of weights) that a tile of 32 tm rows loads, in any order."""
    kept, end = (3 if tm == 1 else 2), (k + 63) // 64
    x, w = {0, 1 if kept == 3 else 0, kept - 1}, {0, 1}
    for s in range(end - 1):
        x.add(s + kept)
        if s & 1:
            w.add((s >> 1) + 2)
    return x, w


@pytest.mark.parametrize("down", [False, True])
def test_scalar_offsets_stay_in_their_buffers(down):
    x_at, w_at = _offset("load_x"), _offset("load_w")
    for k in (*range(16, 1040, 16), 2048, 7168, 8208, 1 << 17):
        # x: the rows of a tile (down), or of all tokens of a pass (up); weights: 16 rows at least
        for rows in (1, 2, 3, 31, 32, 33, 64, 65, 96, 97, 128):
            x_bytes, w_bytes = rows * k * 2, 16 * (k // 2) * (1 if down else 2)
            x, w = _stages(k, -(-rows // 32) if down else 1)
            for s in x:
                base = x_at(s=s, x_bytes=x_bytes, k=k)
                assert 0 <= base <= x_bytes and BEYOND >= x_bytes - base
                if s * 64 < k:                                   # lanes within k read what is theirs
                    assert base == s * 128
            for p in w:
                base = w_at(p=p, w_bytes=w_bytes, k=k)
                assert 0 <= base <= w_bytes
                if p * 128 < k:
                    assert base == p * 64


def test_scalar_offsets_of_scales_are_held():
    at = _offset("load_scales")
    for scale_bytes in (4, 64, 1 << 20):
        for base in (0, 3, 4, 64, 1 << 19, 1 << 25):
            assert at(base=base, scale_bytes=scale_bytes) == min(base, scale_bytes)
