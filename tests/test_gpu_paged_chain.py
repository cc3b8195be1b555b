"""The paged attention's calls together, as a drafting step makes them: slots from device lengths,
norms and rotation with the cache write, attention of the new tokens over the cache; the lengths
advance by what spec_commit accepts.  Eager, captured and replayed, and on two streams at once."""
import numpy as np
import pytest

from gpu_util import log
from oracle import paged as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 2.0 ** -24


def bdr():
    import block_draft_readout_amd as m
    return m


class Layer:
    """One attention layer of B requests that get k + 1 tokens a step."""

    def __init__(self, seed, B=5, k=7, hq=8, hkv=2, d=64, page=16, width=12, fp8=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.k, self.hq, self.hkv, self.d, self.page, self.width, self.fp8 = B, k, hq, hkv, d, page, width, fp8
        self.rows = B * (k + 1)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.cached = z(B)
        self.new = torch.full((B,), k + 1, dtype=torch.int32, device="cuda")
        self.table, self.count = z(B, width) - 1, z(B)
        self.free = torch.randperm(B * width, generator=g, device="cuda").int()
        self.top = torch.full((1,), B * width, dtype=torch.int32, device="cuda")
        shape = (B * width, page, hkv, d)
        if fp8:
            self.kc, self.vc = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.scales = [torch.full((hkv,), s, device="cuda") for s in (0.01, 0.02)]
        else:
            self.kc, self.vc = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.scales = [None, None]
        self.w = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
        self.freq = 1e4 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float32) * 2 / d)
        self.x = torch.zeros(self.rows, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
        self.plan = {n: z(s) for n, s in (("query_offsets", B + 1), ("kv_len", B), ("positions", self.rows),
                                          ("slots", self.rows), ("status", 1))}
        self.plan.update(page_count=self.count, free_count=self.top)
        self.out = torch.zeros(self.rows, hq, d, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros_like(self.out)
        self.lse = None
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step(self):
        m, hq, hkv = bdr(), self.hq, self.hkv
        m.spec_slots(self.cached, self.new, self.table, self.count, self.free, self.top, self.page, self.rows,
                     out=self.plan)
        p = self.plan
        m.dspark_qk_norm_rope(self.x[:, :hq], self.x[:, hq:hq + hkv], self.x[:, hq + hkv:], p["positions"], self.freq,
                              q_weight=self.w[0], k_weight=self.w[1], slots=p["slots"], k_cache=self.kc,
                              v_cache=self.vc, k_scale=self.scales[0], v_scale=self.scales[1], q_out=self.q)
        m.dflash_paged_attention(self.q, self.kc, self.vc, self.table, p["query_offsets"], p["kv_len"], causal=False,
                                 k_scale=self.scales[0], v_scale=self.scales[1], out=self.out, workspace=self.ws)

    def values(self, cache, i, b, length):
        t = torch.arange(length, device="cuda")
        c = cache[self.table[b].long()[t // self.page], t % self.page]
        if self.fp8:
            return c.view(torch.float8_e4m3fn).double().cpu().numpy() * self.scales[i].double().cpu().numpy()[:, None]
        return c.double().cpu().numpy()

    def check(self):
        """The attention against the oracle on the cache as it is (its writes have tests of their own)."""
        q = self.q.double().cpu().numpy().reshape(self.B, self.k + 1, self.hq, self.d)
        out = self.out.double().cpu().numpy().reshape(q.shape)
        for b in range(self.B):
            length = int(self.cached[b]) + self.k + 1
            k, v = self.values(self.kc, 0, b, length), self.values(self.vc, 1, b, length)
            assert np.isfinite(k).all() and np.isfinite(v).all()
            ref, _, mass, s = oracle.attention(q[b], k, v, length - self.k - 1, self.d ** -0.5, False, 0)
            rel = 2 * ((self.d + 4) * EPS * s + (length + 70) * EPS)[..., None]
            assert (np.abs(out[b] - ref) <= 1.01 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + rel) * mass)).all()

    def commit(self, g):
        """Lengths advance by the accepted tokens and the bonus, as spec_commit counts them."""
        m, B, k = bdr(), self.B, self.k
        draft = torch.randint(0, 1000, (B, k), generator=g, device="cuda").int()
        accepted = torch.randint(0, k + 1, (B,), generator=g, device="cuda").int()
        res = m.spec_commit(draft, accepted, draft[:, 0].contiguous())
        lengths = res["row_offsets"][1:] - res["row_offsets"][:-1]
        assert torch.equal(lengths, accepted + 1)
        self.cached.add_(lengths)

    def state(self):
        return [self.table, self.count, self.free, self.top, self.kc, self.vc, self.q, self.out, self.cached, self.x,
                *self.plan.values()]


@pytest.mark.parametrize("fp8", [False, True])
def test_steps(fp8):
    layer = Layer(1, fp8=fp8)
    g = torch.Generator(device="cuda").manual_seed(2)
    for step in range(15):
        layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
        layer.step()
        assert int(layer.plan["status"]) == 0
        if step in (0, 1, 7, 14):
            layer.check()
        layer.commit(g)


def test_steps_captured_and_replayed():
    """Every replay equals the eager step on a copy of its state, with eager work between them."""
    layer, twin = Layer(3, page=4, width=40), Layer(3, page=4, width=40)
    g = torch.Generator(device="cuda").manual_seed(4)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        layer.step()      # once outside: modules are loaded
    stream.synchronize()
    for a, b in zip(layer.state(), twin.state()):
        a.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.step()
    for step in range(12):
        x = torch.randn(layer.x.shape, generator=g, device="cuda")
        layer.x.copy_(x)
        twin.x.copy_(x)
        graph.replay()
        twin.step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(layer.state(), twin.state())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (step, i)
        if step == 5:   # (before the lengths advance)
            twin.check()
        layer.commit(torch.Generator(device="cuda").manual_seed(step))
        twin.commit(torch.Generator(device="cuda").manual_seed(step))


def test_two_graphs_share_a_workspace():
    a, b = Layer(5, width=20), Layer(6, B=3, hq=4, d=128, width=30)
    b.ws = a.ws
    a.new.fill_(8), b.new.fill_(8)
    a.cached.fill_(200), b.cached.fill_(300)
    want = []
    for layer in (a, b):
        layer.x.normal_()
        layer.kc.normal_(), layer.vc.normal_()
        layer.step()
        want.append(layer.out.clone())
    graphs = []
    for layer in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.step()
    for _ in range(3):
        for layer, graph, w in zip((a, b), graphs, want):
            layer.out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_two_streams_at_once():
    layers = [Layer(i, B=6, k=8, hq=16, hkv=4, d=128, width=300) for i in (7, 8)]
    want = []
    for layer in layers:
        layer.cached.fill_(4000)
        layer.x.normal_()
        layer.kc.normal_(), layer.vc.normal_()
        layer.step()
        want.append(layer.out.clone())
        layer.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for s, layer in zip(streams, layers):
            with torch.cuda.stream(s):
                layer.step()
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        assert torch.equal(layer.out, w)


def test_context_rows_without_queries():
    """Keys and values of accepted target positions enter the cache before a block is drafted over
    them; the block's own follow, its tokens see one another."""
    log("context, then block")
    m, layer = bdr(), Layer(9, B=4, k=7, hq=4, d=128)
    g = torch.Generator(device="cuda").manual_seed(10)
    n = torch.tensor([50, 3, 77, 1], dtype=torch.int32, device="cuda")
    rows = int(n.sum())
    plan = m.spec_slots(layer.cached, n, layer.table, layer.count, layer.free, layer.top, layer.page, rows + 9)
    layer.count.copy_(plan["page_count"])
    layer.top.copy_(plan["free_count"])
    kv = torch.randn(rows + 9, 2, layer.hkv, layer.d, generator=g, device="cuda").bfloat16()
    q, k = m.dspark_qk_norm_rope(None, kv[:, 0], kv[:, 1], plan["positions"], layer.freq, q_weight=layer.w[0],
                                 k_weight=layer.w[1], slots=plan["slots"], k_cache=layer.kc, v_cache=layer.vc)
    assert q is None and k is None
    layer.cached.add_(n)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.step()
    assert int(layer.plan["status"]) == 0
    layer.check()
