"""Captured and replayed steps of the paged attention whose row tiles several workgroups share: partials and
records lie in the workspace, and nothing of an earlier replay, of another graph or of the workspace's contents
may reach an output."""
import pytest

from gpu_util import log
from test_gpu_paged_chain import Layer, bdr

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# few rows in one tile and in three, row tiles of 128 and of 256; e4m3
KINDS = {
    "few": dict(B=5, k=7, hq=8, hkv=2, d=64),
    "e4m3": dict(B=4, k=8, hq=10, hkv=2, d=128, fp8=True),
    "128": dict(B=3, k=24, hq=8, hkv=2, d=128),
    "256": dict(B=2, k=79, hq=8, hkv=2, d=128),
}
WIDTH = 200   # pages of 16: past what one launch takes


def _layer(seed, kind):
    layer = Layer(seed, width=WIDTH, **KINDS[kind])
    need = bdr().lib().dflash_paged_attention_workspace_bytes(layer.rows, layer.hq, layer.hkv, layer.d, 1, layer.B,
                                                              WIDTH, layer.page)
    assert need > 0
    layer.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    for c in (layer.kc, layer.vc):
        if layer.fp8:
            c.copy_(torch.randn(c.shape, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            c.normal_(generator=g)
    layer.x.normal_(generator=g)
    layer.cached.fill_(WIDTH * 16 - layer.k - 1)   # once at full length: every request has its pages
    layer.step()
    assert int(layer.plan["status"]) == 0
    return layer


def _graph(layer):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    return graph


def _lengths(layer, i):
    """Cached tokens of the i-th step: long and short by turns, some of them none."""
    top = WIDTH * 16 - layer.k - 1
    some = [top, 17, 0, top // 2, 300, 1, top - 5, 900, 64, 2047]
    return torch.tensor([some[(i * 3 + b * 7) % len(some)] for b in range(layer.B)], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", list(KINDS))
def test_replays_over_changing_lengths(kind):
    log(f"replays over changing lengths: {kind}")
    layer, twin = _layer(1, kind), _layer(1, kind)
    graph = _graph(layer)
    for i in range(8):
        lengths = _lengths(layer, i)
        for one in (layer, twin):
            one.cached.copy_(lengths)
            one.out.fill_(7)
        twin.ws.fill_(255 if i % 2 else 0)   # any contents will do
        if i % 3 == 2:
            layer.ws.fill_(255)
        graph.replay()
        twin.step()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, twin.out), i
        if i in (0, 3):
            layer.check()


@pytest.mark.parametrize("kinds", [("few", "256"), ("e4m3", "128"), ("few", "e4m3")])
def test_graphs_that_share_a_workspace(kinds):
    log(f"graphs that share a workspace: {kinds}")
    layers, twins = [_layer(i, k) for i, k in enumerate(kinds)], [_layer(i, k) for i, k in enumerate(kinds)]
    for layer in layers:
        layer.ws = max((one.ws for one in layers), key=torch.Tensor.numel)
    graphs = [_graph(layer) for layer in layers]
    for i in range(6):
        for layer, twin, graph in zip(layers, twins, graphs):
            lengths = _lengths(layer, i + layer.B)
            for one in (layer, twin):
                one.cached.copy_(lengths)
                one.out.fill_(7)
            graph.replay()
        for twin in twins:
            twin.step()
        torch.cuda.synchronize()
        for layer, twin in zip(layers, twins):
            assert torch.equal(layer.out, twin.out), i
        if i == 2:
            for layer in layers:
                layer.check()
