"""The largest sizes the packed products take, without a GPU: what is beyond
them is refused before any HIP call."""
import os

import pytest

import nvfp4_post_quantization_amd as nq

SHAPE, ALIGN, WS = 2, 3, 4
P = 0x10000                 # never dereferenced
TOKENS = (1 << 31) - 256    # at most
OUT = (1 << 31) - 16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nq.LIB_PATH):
        pytest.skip("libnvfp4mi.so not built")
    return nq.load()


def _calls(lib):
    """The three products as functions of tokens, out_features, y and the workspace's size."""
    return [lambda t, o, y, n: lib.mxfp4_matmul(P, P, t, 32, P, P, o, y, o, P, n, None),
            lambda t, o, y, n: lib.nvfp4_matmul_w4a16(P, t, 32, 32, P, P, P, o, y, o, P, n, None),
            lambda t, o, y, n: lib.nvfp4_matmul_w4a4(P, P, P, t, 32, P, P, P, o, y, o, P, n, None)]


def test_tokens_and_outputs_at_their_limits(lib):
    """Accepted sizes are shown by the error of a misaligned y, which is looked
    for after them."""
    for call in _calls(lib):
        assert call(TOKENS, 4, P + 1, 1 << 40) == ALIGN
        assert call(TOKENS + 1, 4, P + 1, 1 << 40) == SHAPE
        assert call((1 << 31) - 1, 4, P + 1, 1 << 40) == SHAPE
        assert call(20, OUT, P + 1, 1 << 40) == ALIGN
        assert call(20, OUT + 1, P + 1, 1 << 40) == SHAPE


def test_tiles_are_used_where_their_launch_holds(lib):
    """A tile of 256 x 256 has 512 threads and a launch fewer than 2^32: of up
    to 256 tokens, 2^31 - 256 outputs are the last in tiles.  k is off the
    stages' length there, so that tiles need a workspace (of scales copied to
    rows of words) and the streaming kernels none."""
    for q, k in ((lib.mxfp4_matmul_workspace_bytes, 32), (lib.nvfp4_matmul_workspace_bytes, 16)):
        for t in (33, 100, 128, 129, 256):
            assert q(t, (1 << 31) - 256, k) >= 4 * ((1 << 31) - 256)
            assert q(t, (1 << 31) - 255, k) == 0
            assert q(t, OUT, k) == 0
        for o in (1, 100, 256):
            assert q(TOKENS, o, k) > 0
        assert q(257, (1 << 30) - 256, k) > 0 and q(257, 1 << 30, k) == 0


def test_tiles_of_few_tokens_are_not_the_large_ones(lib):
    """Up to 128 tokens fill one row of small tiles, and half a large one at
    most, however many outputs there are.  Small tiles show by the channel
    parts that this many of them are split into, whose sums need a workspace."""
    k = 1 << 18                                     # enough that parts pay: 1 part 1.4 x 2048 stages, 4 parts 3/4 of that
    for q, own in ((lib.mxfp4_matmul_workspace_bytes, 0),
                   (lib.nvfp4_matmul_workspace_bytes, 2)):                  # bytes of W4A4's activations a channel
        for t in (33, 128):
            assert q(t, 49152, k) - own * t * k >= 2 * t * 49152 * 4
            # where small tiles might be more than a launch holds: no parts, no sums
            assert q(t, 1 << 26, 2048) == own * t * 2048
        assert q(129, 49152, k) == own * 129 * k


def test_too_little_workspace_at_the_limit(lib):
    for call, q in zip(_calls(lib), (lib.mxfp4_matmul_workspace_bytes, lib.nvfp4_matmul_workspace_bytes,
                                     lib.nvfp4_matmul_workspace_bytes)):
        n = q(100, (1 << 31) - 256, 32)
        assert n and call(100, (1 << 31) - 256, P, n - 1) == WS
