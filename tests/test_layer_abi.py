"""CPU tests of the convolution's, the scan's and the norm's entry points: the
host code under the sanitizers (every refusal and size query of the C ABI),
the sizes the binding and the kernels agree on, and the checks the PyTorch
wrappers make before a pointer leaves Python."""
import ctypes
import os
import shutil
import subprocess

import pytest

from gated_delta_rule_recurrence_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_recurrence_amd", "csrc")
BUILD = os.path.join(CSRC, "_build")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"


@pytest.fixture(scope="module")
def lib():
    if not _lib.LIB_PATH.exists():
        from gated_delta_rule_recurrence_amd import build
        build.build(verbose=False)
    return _lib.load()


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="ROCm compilers not installed")
def test_host_code_under_asan_ubsan(tmp_path):
    from gated_delta_rule_recurrence_amd import build
    need = os.path.join(BUILD, "gdr_layer_api.o")
    if not os.path.exists(need):
        build.build(verbose=False)
    objs = [os.path.join(BUILD, f) for f in sorted(os.listdir(BUILD))
            if f.endswith(".o") and f != "gdr_layer_api.o"]
    inc = os.path.join(ROOT, "include")
    api, drv, exe = (tmp_path / n for n in ("layer_api_san.o", "layer_host_check.o", "layer_host_check"))
    run = lambda cmd: subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    # sanitizers on the host pass only (the device code is built as usual)
    r = run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             f"-I{inc}", "-c", os.path.join(CSRC, "gdr_layer_api.hip"), "-o", str(api)])
    assert r.returncode == 0, r.stderr
    r = run([CLANG, "-g", "-O1", "-fno-gpu-sanitize", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", f"-I{inc}", "-c",
             os.path.join(ROOT, "tests", "layer_host_check.c"), "-o", str(drv)])
    assert r.returncode == 0, r.stderr
    r = run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", str(drv), str(api), *objs, "-o", str(exe)])
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
    assert "layer host checks passed" in out


def test_structures_match_the_header(lib):
    """A size query reads the last field of each structure: a wrong layout
    would reject, or accept, the wrong value."""
    conv = _lib.GdrConvShape(1, 8, 8, 16, 4, 0, 0, 0, 1, 0)
    assert _lib.size_of("gdr_conv_backward_workspace_bytes", conv) > 0
    conv.act = 5
    with pytest.raises(_lib.GdrError, match="act"):
        _lib.size_of("gdr_conv_backward_workspace_bytes", conv)
    scan = _lib.GdrScanShape(1, 8, 8, 16, 4, 1, 0, 0, 0, 0, 0, 0, 1)
    assert _lib.size_of("gdr_scan_checkpoint_bytes", scan) > 0
    scan.softplus = 5
    with pytest.raises(_lib.GdrError, match="softplus"):
        _lib.size_of("gdr_scan_checkpoint_bytes", scan)
    norm = _lib.GdrNormShape(8, 16, 4, 0, 0, 1e-6, 0, 0, 0, 0, 1)
    assert _lib.size_of("gdr_norm_backward_workspace_bytes", norm) > 0
    norm.act = 5
    with pytest.raises(_lib.GdrError, match="act"):
        _lib.size_of("gdr_norm_backward_workspace_bytes", norm)
    assert ctypes.sizeof(conv) == 6 * 8 + 16
    assert ctypes.sizeof(scan) == 11 * 8 + 8
    assert ctypes.sizeof(norm) == 5 * 8 + 24


@pytest.mark.parametrize("B,T,C,N", [(1, 2048, 4096, 16), (4, 4096, 4096, 16), (2, 100, 40, 40), (3, 1, 64, 5)])
def test_scan_save_buffer(lib, B, T, C, N):
    """A state every 8 steps (4 for N > 16), states
    padded to a power of two, a slot per sequence and one more to spare."""
    s = _lib.GdrScanShape(B, T, B * T, C, N, 1, 0, 0, 0, 0, 0, 1, 1)
    pad = 4
    while pad < N:
        pad *= 2
    tile = 8 if N <= 16 else 4
    assert _lib.size_of("gdr_scan_checkpoint_bytes", s) == C * pad * 4 * (B * T // tile + B + 1)


# ---- what the wrappers refuse ----------------------------------------------------

def test_rows_and_strides():
    import torch
    from gated_delta_rule_recurrence_amd import ops
    cpu = torch.device("cpu")
    f = lambda t, tail, **k: ops._row_stride("x", t, tail, torch.float32, cpu, **k)
    x = torch.zeros(2, 5, 12)
    assert f(x, (12,)) == (10, 12)
    assert f(x[..., 4:8], (4,)) == (10, 12)
    assert f(x[:, :, :8].unflatten(-1, (2, 4)), (2, 4)) == (10, 12)
    assert f(x[:1], (12,)) == (5, 12)
    assert f(x[:, :1], (12,)) == (2, 60)
    assert f(x[:0], (12,)) == (0, 12)
    assert f(torch.zeros(10, 12), (12,)) == (10, 12)
    for bad, tail in ((x[:, :3], (12,)), (x.transpose(0, 1), (12,)), (x[..., ::2], (6,)), (x, (11,)),
                      (x[:, :, :8].unflatten(-1, (2, 4)).transpose(2, 3), (4, 2)), (torch.zeros(12), (12,)),
                      (torch.zeros(12).expand(3, 12), (12,))):
        with pytest.raises(ValueError):
            f(bad, tail)
    with pytest.raises(ValueError, match="rows"):
        f(x, (12,), rows=9)
    with pytest.raises(ValueError, match="dtype"):
        f(x.double(), (12,))
    with pytest.raises(TypeError):
        f(None, (12,))


def test_sequences():
    import torch
    from gated_delta_rule_recurrence_amd import ops
    cpu = torch.device("cpu")
    x = torch.zeros(2, 5, 12)
    assert ops._sequences(x, 10, (12,), None, None, cpu) == (2, 5)
    assert ops._sequences(x, 10, (12,), None, 2, cpu) == (5, 2)
    assert ops._sequences(x[:, :0], 0, (12,), None, 0, cpu) == (2, 0)
    assert ops._sequences(torch.zeros(0, 12), 0, (12,), None, 0, cpu) == (0, 0)
    for rows, T in ((10, 3), (10, 0), (10, -1)):
        with pytest.raises(ValueError):
            ops._sequences(x, rows, (12,), None, T, cpu)
    with pytest.raises(ValueError, match="T is needed"):
        ops._sequences(x.view(10, 12), 10, (12,), None, None, cpu)
    with pytest.raises(ValueError, match="act"):
        ops._act("relu")


def test_cpu_tensors_are_refused():
    import torch
    from gated_delta_rule_recurrence_amd import ops
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ops.gdr_conv_forward(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        ops.gdr_norm_forward(x, groups=2)
    with pytest.raises(ValueError, match="GPU"):
        ops.gdr_scan_forward(x, x, torch.zeros(8, 2), torch.zeros(1, 4, 1, 2), torch.zeros(1, 4, 1, 2))
