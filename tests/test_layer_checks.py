"""CPU tests of what the convolution's, the scan's and the norm's entry points
check before anything is launched: buffers that a caller hands over, and
tensors that overlap.  No GPU is involved: the launch is replaced, or the call
is refused on the host."""
import pytest

from gated_delta_rule_recurrence_amd import _lib


@pytest.fixture(scope="module")
def lib():
    if not _lib.LIB_PATH.exists():
        from gated_delta_rule_recurrence_amd import build
        build.build(verbose=False)
    return _lib.load()


@pytest.fixture
def on_cpu(lib, monkeypatch):
    """The wrappers with CPU tensors let through and calls listed instead of
    launched."""
    from gated_delta_rule_recurrence_amd import ops
    calls = []
    monkeypatch.setattr(ops, "_gpu", lambda x: (x.device, x.dtype))
    monkeypatch.setattr(ops, "_launch", lambda name, *rest: calls.append(name))
    return calls


def scan_rows(T, C=64, N=16):
    import torch
    x = torch.zeros(1, T, C)
    return x, x, torch.zeros(C, N), torch.zeros(1, T, 1, N), torch.zeros(1, T, 1, N), None, None, None


def test_scan_backward_checks_the_saved_buffer(on_cpu):
    """More rows than the forward had, or a buffer that is not the forward's:
    the kernel would read the saved states of all rows."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    few, many = scan_rows(16), scan_rows(400)
    _, _, saved = ops.gdr_scan_forward(*few)
    ops.gdr_scan_backward(*few, saved, few[0])
    assert on_cpu == ["gdr_scan_forward", "gdr_scan_backward"]
    saved.T = 400
    with pytest.raises(ValueError, match="saved.ckpt too small"):
        ops.gdr_scan_backward(*many, saved, many[0])
    _, _, saved = ops.gdr_scan_forward(*many)
    saved.ckpt = saved.ckpt[:-1]
    with pytest.raises(ValueError, match="saved.ckpt too small"):
        ops.gdr_scan_backward(*many, saved, many[0])
    saved.ckpt = torch.zeros(2 * len(saved.ckpt) + 2, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError, match="saved.ckpt must be contiguous"):
        ops.gdr_scan_backward(*many, saved, many[0])
    saved.ckpt = None
    with pytest.raises(TypeError, match="saved.ckpt"):
        ops.gdr_scan_backward(*many, saved, many[0])
    assert on_cpu[2:] == ["gdr_scan_forward"]


# ---- rows over rows (never launched: refused calls only, at made-up addresses) -----

X, FAR = 1 << 20, 1 << 40


def conv_shape(B, T, C, stride=0, bf16=False, K=4):
    dt = _lib.GDR_BF16 if bf16 else _lib.GDR_F32
    return _lib.GdrConvShape(B, T, B * T, C, K, stride, dt, dt, _lib.GDR_ACT_SILU, 0)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,T,C,stride,x,y", [
    (2, 17, 32, 0, X, X),              # in place, more than one tile
    (1, 16, 32, 40, X, X),             # one tile, but not the same rows
    (1, 16, 32, 0, X, X + 16),         # one tile, shifted
    (1, 40, 32, 0, X + 16, X),
    (1, 40, 32, 0, X, X + 40 * 64 - 16),   # the last bytes of either type
    (1, 40, 32, 0, X + 40 * 64 - 16, X),
    (2, 40, 32, 512, X, X + 512),      # dense rows that run into x's next ones
])
def test_conv_refuses_rows_over_rows(lib, B, T, C, stride, x, y, bf16):
    s = conv_shape(B, T, C, stride, bf16)
    far = [FAR + (k << 30) for k in range(8)]
    assert _lib.layer_raw("gdr_conv_forward", s, (x, far[0], far[1], 0, 0, y, 0), 0) == _lib.GDR_ERR_OVERLAP
    assert "overlap" in _lib.strerror(_lib.GDR_ERR_OVERLAP)
    n = _lib.size_of("gdr_conv_backward_workspace_bytes", s)
    ptrs = lambda x, dy, dx: (x, far[0], far[1], 0, 0, dy, 0, dx, far[2], far[3], 0, far[4])
    assert _lib.layer_raw("gdr_conv_backward", s, ptrs(x, far[5], y), 0, n) == _lib.GDR_ERR_OVERLAP
    if stride == 0:
        assert _lib.layer_raw("gdr_conv_backward", s, ptrs(far[5], x, y), 0, n) == _lib.GDR_ERR_OVERLAP


# ---- partial sums of packed rows ---------------------------------------------------

PACKS = [(64, 65536, 65536), (1000, 65536, 65536), (7, 6000, 6000), (64, 65536, 4096), (3, 300, 2 ** 30 - 1),
         (5, 0, 300), (5, 300, 0), (1, 1, 300), (4, 2048, 512)]


@pytest.mark.parametrize("B,rows,T", PACKS)
def test_conv_partial_sums_follow_the_rows(lib, B, rows, T):
    """B sequences of packed rows, T at most the longest (all rows, where
    nobody says): one partial sum of dweight and dbias for every started piece
    of at least 64 steps, of which disjoint sequences have rows / 64 + B at
    most, whatever T is."""
    C, K = 14336, 4
    s = _lib.GdrConvShape(B, T, rows, C, K, 0, _lib.GDR_BF16, _lib.GDR_BF16, _lib.GDR_ACT_SILU, 0)
    n = _lib.size_of("gdr_conv_backward_workspace_bytes", s)
    assert 0 < n <= (rows // 64 + B) * (K + 1) * C * 4


@pytest.mark.parametrize("B,rows,T", PACKS)
@pytest.mark.parametrize("C,N,G", [(4096, 16, 1), (2048, 64, 2), (100, 5, 4)])
def test_scan_partial_sums_follow_the_rows(lib, B, rows, T, C, N, G):
    """The same for the scan's dA, dD and ddt_bias: a partial sum for every
    started chunk (16 steps at least), as the states between chunks have it."""
    s = _lib.GdrScanShape(B, T, rows, C, N, G, 0, 0, 0, 0, 0, _lib.GDR_BF16, 1)
    pad = next(p for p in (4, 8, 16, 32, 64) if p >= N)
    pieces = rows // 16 + B + 1
    tiles = -(-C // G // 64)  # dB, dC: one of each a tile of 64 channels
    most = pieces * C * (pad + 2) * 4 + pieces * C * (pad + 1) * 4 + rows * 8 * G * N * tiles + 4 * 256
    assert _lib.size_of("gdr_scan_backward_workspace_bytes", s) <= most
