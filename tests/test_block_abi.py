"""CPU tests of linear attention's and the block norms' entry points: the host
code under the sanitizers (every refusal and size query of the C ABI), the
structures the binding shares with the header, and the checks that the PyTorch
wrappers make before a pointer leaves Python."""
import os
import subprocess

import pytest

from gated_delta_rule_recurrence_amd import _lib
from tests.test_layer_abi import BUILD, CLANG, CSRC, HIPCC, ROOT, lib  # noqa: F401
from tests.test_layer_checks import on_cpu  # noqa: F401


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="ROCm compilers not installed")
def test_host_code_under_asan_ubsan(tmp_path):
    from gated_delta_rule_recurrence_amd import build
    if not os.path.exists(os.path.join(BUILD, "gdr_layer_api.o")):
        build.build(verbose=False)
    objs = [os.path.join(BUILD, f) for f in sorted(os.listdir(BUILD)) if f.endswith(".o") and f != "gdr_layer_api.o"]
    inc = os.path.join(ROOT, "include")
    api, drv, exe = (tmp_path / n for n in ("layer_api_san.o", "block_host_check.o", "block_host_check"))
    run = lambda cmd: subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    # sanitizers on the host pass only (the device code is built as usual)
    r = run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             f"-I{inc}", "-c", os.path.join(CSRC, "gdr_layer_api.hip"), "-o", str(api)])
    assert r.returncode == 0, r.stderr
    r = run([CLANG, "-g", "-O1", "-fno-gpu-sanitize", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", f"-I{inc}", "-c",
             os.path.join(ROOT, "tests", "block_host_check.c"), "-o", str(drv)])
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
    assert "block host checks passed" in out


def test_structures_match_the_header(lib):  # noqa: F811
    """A size query reads the last field of each structure: a wrong layout
    would reject, or accept, the wrong value."""
    lin = _lib.GdrLinShape(1, 200, 200, 2, 4, 64, 64, 0, 0, 0, 0, 1.0, 1, 0, 0)
    assert _lib.size_of("gdr_lin_backward_workspace_bytes", lin) > 0
    lin.per_head = 5
    with pytest.raises(_lib.GdrError, match="per_head"):
        _lib.size_of("gdr_lin_checkpoint_bytes", lin)
    res = _lib.GdrResShape(8, 16, 0, 0, 0, 0, 1.0, 1e-6, 0.0, 0, 0, 0, 0, 1, 1, 0)
    assert _lib.size_of("gdr_res_backward_workspace_bytes", res) > 0
    res.center = 5
    with pytest.raises(_lib.GdrError, match="center"):
        _lib.size_of("gdr_res_backward_workspace_bytes", res)


def test_limits_match_the_header(lib):  # noqa: F811
    text = open(os.path.join(ROOT, "include", "gdr.h")).read()
    assert f"#define GDR_LIN_MAX_DIM {_lib.LIN_MAX_DIM}\n" in text
    assert f"#define GDR_RES_MAX_CHANNELS {_lib.RES_MAX_CHANNELS}\n" in text


def test_workspaces_follow_the_rows(lib):  # noqa: F811
    """Many short sequences whose T is not stated need no more than their rows
    do: the states around segments are numbered through the rows."""
    def shape(B, T, rows):
        return _lib.GdrLinShape(B, T, rows, 16, 16, 128, 128, 0, 0, 0, 0, 1.0, 1, 0, 0)
    state = 16 * 128 * 128 * 4
    one = _lib.size_of("gdr_lin_checkpoint_bytes", shape(1, 65536, 65536))
    many = _lib.size_of("gdr_lin_checkpoint_bytes", shape(1000, 65536, 65536))
    assert one < many <= one + 2 * 999 * state
    # single tokens into a large buffer: two states a sequence
    assert _lib.size_of("gdr_lin_checkpoint_bytes", shape(4, 1, 65536)) <= 10 * state


def test_lin_buffers_are_checked(on_cpu):  # noqa: F811
    import torch
    from gated_delta_rule_recurrence_amd import ops
    q, v = torch.zeros(1, 300, 2, 16), torch.zeros(1, 300, 4, 16)
    lg = torch.zeros(1, 300, 4)
    _, _, saved = ops.gdr_lin_forward(q, q, v, lg)
    ops.gdr_lin_backward(q, q, v, lg, saved, v)
    assert on_cpu == ["gdr_lin_forward", "gdr_lin_backward"]
    for bad, match in ((saved.ckpt[:-1], "too small"), (torch.zeros(2 * len(saved.ckpt) + 2, dtype=torch.uint8)[::2], "contiguous")):
        with pytest.raises(ValueError, match=match):
            ops.gdr_lin_backward(q, q, v, lg, ops.LinSaved(bad, None, 300, 1.0), v)
    with pytest.raises(TypeError, match="saved.ckpt"):
        ops.gdr_lin_backward(q, q, v, lg, ops.LinSaved(None, None, 300, 1.0), v)
    with pytest.raises(ValueError, match="workspace too small"):
        ops.gdr_lin_backward(q, q, v, lg, saved, v, workspace=torch.zeros(8, dtype=torch.uint8))
    for bad in (lambda: ops.gdr_lin_forward(q, q[:, :1], v, lg), lambda: ops.gdr_lin_forward(q, q, v, lg[..., :2]),
                lambda: ops.gdr_lin_forward(q, q, v, lg, torch.zeros(1, 4, 16, 15)),
                lambda: ops.gdr_lin_forward(q[0, 0], q, v), lambda: ops.gdr_lin_forward(q, q, v[0, 0, 0]),
                lambda: ops.gdr_lin_forward(q, q, v, torch.zeros(3)),
                lambda: ops.gdr_lin_forward(q[0], q[0], v[0], spans=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    assert len(on_cpu) == 2


def test_res_gates(on_cpu, monkeypatch):  # noqa: F811
    """Which rows of x a gate's row serves, by its shape."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    seen = []
    monkeypatch.setattr(ops, "_launch", lambda name, shape, *rest: seen.append(shape.gate_rows))
    x = torch.zeros(3, 5, 8)
    for gate, want in ((None, 0), (torch.zeros(8), 0), (torch.zeros(3, 8), 5), (torch.zeros(3, 1, 8), 5), (torch.zeros(3, 5, 8), 1)):
        ops.gdr_res_forward(x, x, gate)
        assert seen.pop() == want
    ops.gdr_res_forward(x[0], x[0], torch.zeros(5, 8))
    assert seen.pop() == 1
    ops.gdr_res_forward(x[0], x[0], torch.zeros(1, 8))
    assert seen.pop() == 5
    for bad in (torch.zeros(5, 8), torch.zeros(3, 7), torch.zeros(3, 2, 8), torch.zeros(3, 1, 8).expand(3, 5, 8), torch.zeros(3, 8).half(), 2.0):
        with pytest.raises((ValueError, TypeError)):
            ops.gdr_res_forward(x, x, bad)
    assert not seen
