"""Two losses over the same hidden states and head on two streams at once, each with a workspace
of its own.  Both streams wait for the same product on the default stream while all of their calls
are queued, so their kernels start together and run beside each other."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


@pytest.mark.parametrize("dtype,N,H,V,r", [("bf16", 400, 264, 30011, 16), ("bf16", 50, 1032, 30011, 8),
                                           ("bf16", 1200, 520, 20011, 32), ("f32", 130, 132, 10007, 8)])
def test_shared_inputs_in_flight_together(dtype, N, H, V, r):
    import block_draft_readout_amd as m
    from gpu_util import log
    g = torch.Generator(device="cuda").manual_seed(N + V)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w = rn(N, H).to(t), (rn(V, H) * 2 / H ** 0.5).to(t)
    w1, w2 = rn(V, r).to(t), (rn(V, r) * 0.3).to(t)
    prev = torch.randint(-1, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    lab = torch.randint(-V // 5, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.randint(-V // 5, V, (N, 8), generator=g, device="cuda", dtype=torch.int32)
    u, lg = rn(N, 8), torch.rand(N, generator=g, device="cuda") + 0.2
    mk = dict(markov_w1=w1, markov_w2=w2, prev_token=prev)
    L, dt = m.lib(), m.BDR_BF16 if dtype == "bf16" else m.BDR_F32
    ws = [torch.empty(n + 256, dtype=torch.uint8, device="cuda")
          for n in (max(L.dspark_ce_workspace_bytes(N, H, V, r, dt, b) for b in (0, 1)),
                    max(L.dspark_distill_workspace_bytes(N, H, V, r, 8, dt, b) for b in (0, 1)))]

    def ce():
        loss, lse = m.dspark_ce_loss(x, w, lab, workspace=ws[0], **mk)
        yield [loss, lse]
        yield list(m.dspark_ce_backward(x, w, lab, lse, lg, workspace=ws[0], **mk).values())

    def distill():
        loss, lse, picked = m.dspark_distill_loss(x, w, ids, u, temperature=2.0, workspace=ws[1], **mk)
        yield [loss, lse, picked]
        yield list(m.dspark_distill_backward(x, w, ids, u, lse, picked, lg, temperature=2.0,
                                             workspace=ws[1], **mk).values())

    alone = []
    for f in (ce, distill):
        alone.append([o for outs in f() for o in outs])
        torch.cuda.synchronize()
    assert all(bool(o.any()) for a in alone for o in a)
    streams = [torch.cuda.Stream() for _ in range(2)]
    big = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    queued = 0
    for _ in range(4):
        for k in ws:
            k.fill_(255)
        torch.cuda.synchronize()
        gate = torch.cuda.Event()
        for _ in range(16):             # some 10 ms
            big = big @ big
        gate.record()
        got, calls = [[], []], [ce(), distill()]
        for s in streams:
            s.wait_event(gate)
        for _half in range(2):          # forward of both, then backward of both
            for k in range(2):
                with torch.cuda.stream(streams[k]):
                    got[k] += next(calls[k])
        queued += not gate.query()      # everything was queued before anything ran
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert len(a) == len(b)
            for i, (p, q) in enumerate(zip(a, b)):
                assert torch.equal(p, q), i
    log(f"two streams {dtype} {N}: all calls were queued before the first ran {queued} times of 4")
    assert queued
