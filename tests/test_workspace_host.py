"""Sizes that the binding reports for caller-given workspaces: what is left of the tensor past
the next 256-byte boundary, and never below zero (the C ABI takes the size as unsigned)."""
import pytest

torch = pytest.importorskip("torch")


def _slices():
    base = torch.zeros(4096, dtype=torch.uint8)
    to = -base.data_ptr() % 256            # first aligned byte
    for off, n in ((16, 100), (1, 1), (1, 255), (16, 240), (255, 1), (16, 241), (0, 0), (0, 64), (0, 2048),
                   (8, 2048), (16, 16)):
        ws = base[to + off:to + off + n]
        want = max(0, n - (256 - off) % 256) if n else 0
        yield ws, want


def test_training_workspace_sizes():
    from block_draft_readout_amd import training
    for ws, want in _slices():
        p, n, kept = training._space(1 << 20, ws.device, ws)
        assert p % 256 == 0 and n == want and kept is ws, (ws.numel(), ws.data_ptr() % 256, n)


def test_workspace_sizes():
    import block_draft_readout_amd as bdr
    for ws, want in _slices():
        p, n = bdr._ws_ptr(ws)
        assert (p.value or 0) % 256 == 0 and n == want, (ws.numel(), ws.data_ptr() % 256, n)


def test_short_misaligned_workspace_is_refused_by_the_library():
    """The size as the C ABI receives it is below what a call needs."""
    import ctypes
    import os
    from block_draft_readout_amd import _abi, build, training
    if not os.path.exists(_abi.LIB_PATH):
        build.build()
    L = _abi.load()
    ws = next(s for s, _ in _slices())
    p, n, _ = training._space(1 << 20, ws.device, ws)
    P = 1 << 20     # an aligned address; never dereferenced
    need = L.dspark_norm_backward_workspace_bytes(4, 64)
    assert ctypes.c_size_t(n).value < need
    rc = L.dspark_norm_backward(P << 2, 64, P, 64, 4, 64, _abi.BDR_BF16, P, P, P, P << 1, P, P, p, n, None)
    assert rc == _abi.BDR_EWORKSPACE
