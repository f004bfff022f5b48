"""The packed products and the expert layer as a program uses them: chained and
captured, several at once, and with as many jobs as the layer can have."""
import numpy as np
import pytest
import torch

import nvfp4_post_quantization_amd as nq

from _gpu import DEV, need_gpu, note
from test_gpu_product_range import Experts

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def test_layer_of_the_most_jobs():
    """64 tokens, 16 places: every place its own of 1024 experts, and all
    tokens on the same 16."""
    note("layer 1024 jobs")
    L = Experts(1, 64, 64, 48, 1024, 16)
    L.ids = torch.randperm(1024, generator=torch.Generator().manual_seed(0)).view(64, 16).int().to(DEV)
    L.check(L.run())
    L.ids = (torch.arange(16, device=DEV, dtype=torch.int32) * 64 + 63).repeat(64, 1)
    L.check(L.run())


def test_layers_on_two_streams():
    note("layers on two streams")
    layers = [Experts(i, t, 512, 544, 16, 4) for i, t in ((1, 3), (2, 50))]
    want = [L.run().clone() for L in layers]
    ws = [torch.full((nq.moe_workspace_bytes(L.dims[0], 4, 544),), 255, dtype=torch.uint8, device=DEV) for L in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for L, w, s in zip(layers, ws, streams):
            with torch.cuda.stream(s):
                got.append(nq.moe_forward(L.x, L.ids, L.wt, *L.w, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("normalize", [True, False])
def test_captured_route_and_layer(normalize):
    note(f"captured route and layer normalize={normalize}")
    tokens, top_k = 7, 3
    L = Experts(4, tokens, 256, 160, 24, top_k)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    logits = [torch.randn((tokens, 24), generator=g, device=DEV) for _ in range(3)]
    xs = [torch.randn((tokens, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]
    def step(z, x, out, y, ws):
        nq.moe_route(z, top_k, normalize=normalize, out=out)
        nq.moe_forward(x, *out, *L.w, out=y, workspace=ws)
    def buffers():
        return ((torch.empty((tokens, top_k), dtype=torch.int32, device=DEV), torch.empty((tokens, top_k), device=DEV)),
                torch.empty((tokens, 256), dtype=torch.bfloat16, device=DEV),
                torch.empty(nq.moe_workspace_bytes(tokens, top_k, 160), dtype=torch.uint8, device=DEV))
    want = []
    for z, x in zip(logits, xs):
        out, y, ws = buffers()
        step(z, x, out, y, ws)
        want.append((out[0], out[1], y))
    z, x = logits[0].clone(), xs[0].clone()
    out, y, ws = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(z, x, out, y, ws)
    for i in (1, 2, 0, 1):
        z.copy_(logits[i])
        x.copy_(xs[i])
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out[0], out[1], y), want[i]):
            assert torch.equal(a, b)
        step(logits[i], xs[i], *buffers())                           # eager work between replays


@pytest.mark.parametrize("tokens", [5, 100])
def test_captured_quantize_product_dequant(tokens):
    note(f"captured quantize, product, dequant tokens={tokens}")
    k, out = 544, 160
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    w = nq.mxfp4_quantize(torch.randn((out, k), generator=g, device=DEV).to(torch.bfloat16))
    xs = [torch.randn((tokens, k), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]
    def step(x, q, y, back, ws):
        nq.mxfp4_quantize(x, out=q)
        nq.mxfp4_matmul(*q, *w, out=y, workspace=ws)
        nq.mxfp4_dequant(*q, out=back)
    def buffers():
        return ((torch.empty((tokens, k // 2), dtype=torch.uint8, device=DEV),
                 torch.empty((tokens, k // 32), dtype=torch.uint8, device=DEV)),
                torch.empty((tokens, out), dtype=torch.bfloat16, device=DEV),
                torch.empty((tokens, k), dtype=torch.bfloat16, device=DEV),
                torch.empty(max(nq.mxfp4_matmul_workspace_bytes(tokens, out, k), 1), dtype=torch.uint8, device=DEV))
    want = []
    for x in xs:
        b = buffers()
        step(x, *b)
        want.append((*b[0], b[1], b[2]))
    x, b = xs[0].clone(), buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, *b)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        b[3].fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for a, r in zip((*b[0], b[1], b[2]), want[i]):
            assert torch.equal(a, r)
        step(xs[i], *buffers())
