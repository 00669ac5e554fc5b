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
