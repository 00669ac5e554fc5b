"""GPU tests of the convolution, the scan and the norm at their edges:
infinities beside the steps that pad a tile, steps that change nothing,
outputs over inputs, partial sums of packed rows, the measurement hook."""
import numpy as np
import pytest

import oracle.layer_oracle as L
from test_gpu_layer_ops import ARGS, F32, GRADS, check, dev_of, same, scan_inputs, small_state

pytestmark = pytest.mark.gpu


# ---- scan: the steps that pad a sequence's last tile ------------------------------

@pytest.mark.parametrize("T", [1, 3, 21, 24, 150, 152])
def test_infinite_rates_backward(cuda, T):
    """A = -inf is what the lowest finite rates are, in every gradient: the
    adjoint of the last state passes the padding steps, whose decay is 1."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    u, dt, A, Bm, Cm, D, z, bias, S0 = small_state(cuda)["scan"]
    u, dt, Bm, Cm, z = [t[:, :T].contiguous() for t in (u, dt, Bm, Cm, z)]
    dy = small_state(cuda)["dy"][:, :T].contiguous()
    dS_T = 3 * torch.randn(S0.shape, device=cuda, generator=torch.Generator(device=cuda).manual_seed(1))
    got = []
    for rate in (-float("inf"), -1e30):
        A = A.clone()
        A[::3] = rate
        args = u, dt, A, Bm, Cm, D, z, bias
        y, S_T, saved = ops.gdr_scan_forward(*args, S0)
        grads = ops.gdr_scan_backward(*args, saved, dy, dS_T)
        for name, g in zip(GRADS, grads):
            assert torch.isfinite(g).all(), name
        got.append([y, S_T, *grads])
    assert same(*got)


@pytest.mark.parametrize("N", [1, 7, 16, 24, 40])
@pytest.mark.parametrize("T", [1, 3, 21, 24, 150, 152])
def test_an_infinite_last_input(cuda, N, T):
    """u = inf in the last step makes the last state infinite.  dA, dS0, du
    and the earlier ddt do not depend on that state and are those of the
    formula; ddt of the last step and its sum are infinite, not NaN."""
    from gated_delta_rule_recurrence_amd import ops
    C, B = 40, 2
    p = scan_inputs("f32", B, B * T, C, N, 1, T)
    for b in range(B):
        p["u"][(b + 1) * T - 1, 3::5] = np.inf
    d = {k: dev_of(v, "f32", cuda) for k, v in p.items()}
    d = {k: v.view(B, T, *v.shape[1:]) if k not in F32 else v for k, v in d.items()}
    _, _, saved = ops.gdr_scan_forward(*[d[k] for k in ARGS])
    got = dict(zip(GRADS, ops.gdr_scan_backward(*[d[k] for k in ARGS[:8]], saved, d["dy"], d["dS_T"])))
    args = [p[k] for k in ARGS] + [True, [(b * T, (b + 1) * T) for b in range(B)]]
    with np.errstate(invalid="ignore"):
        ref, mag = (L.scan_backward(*args, p["dy"], p["dS_T"], mag=m) for m in (False, True))
    n = 2 * (128 + 4 * T)
    check("dA", got["dA"], ref["dA"], mag["dA"], "f32", n + B * T)
    check("dS0", got["dS0"], ref["dS0"], mag["dS0"], "f32", n)
    check("du", got["du"], ref["du"], mag["du"], "f32", n + 128)
    ddt = got["ddt"].double().cpu().numpy().reshape(B * T, C)
    finite = np.isfinite(ref["ddt"])
    assert finite.sum() == B * (T * C - 8) and (ddt[~finite] == ref["ddt"][~finite]).all()
    off = np.abs(ddt[finite] - ref["ddt"][finite])
    assert (off <= (n + 129) * 2.0 ** -24 * mag["ddt"][finite]).all()
    total, want = got["ddt_bias"].double().cpu().numpy(), ref["ddt_bias"]
    assert (np.isinf(total) | np.isnan(want))[3::5].all() and np.isfinite(np.delete(total, np.s_[3::5])).all()
    assert (total[np.isinf(want)] == want[np.isinf(want)]).all()


# ---- scan: a step of delta = 0 -----------------------------------------------------

@pytest.mark.parametrize("T", [1, 4, 5, 40])
@pytest.mark.parametrize("N", [3, 16, 33])
@pytest.mark.parametrize("softplus", [False, True])
def test_no_step_keeps_the_state(cuda, T, N, softplus):
    """delta = 0 is an identity step whatever the rate, A = -inf too, in the
    kernel of few steps as in the tiled one: S_T is S0 and y reads it."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    C, B = 70, 2
    g = torch.Generator(device=cuda).manual_seed(T)
    S0 = torch.randn(B, C, N, device=cuda, generator=g)
    A = -torch.exp(torch.randn(C, N, device=cuda, generator=g))
    A[::3] = -float("inf")
    u, Cm = torch.randn(B, T, C, device=cuda, generator=g), torch.randn(B, T, 1, N, device=cuda, generator=g)
    # (e^-200 is 0 in 32 bits)
    dt = torch.full((B, T, C), -200.0 if softplus else 0.0, device=cuda)
    y, S_T, _ = ops.gdr_scan_forward(u, dt, A, Cm, Cm, S0=S0, softplus=softplus)
    assert torch.equal(S_T, S0)
    ref = torch.einsum("btn,bcn->btc", Cm[:, :, 0].double().cpu(), S0.double().cpu())
    mag = torch.einsum("btn,bcn->btc", Cm[:, :, 0].double().cpu().abs(), S0.double().cpu().abs())
    assert ((y.double().cpu() - ref).abs() <= (N + 4) * 2.0 ** -24 * mag).all()


# ---- convolution: y over x ---------------------------------------------------------

@pytest.mark.parametrize("dtype,C", [("bf16", 2056), ("bf16", 33), ("f32", 1500)])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_conv_over_its_input(cuda, dtype, C, T):
    """Up to 16 steps y may be x; more are refused, and so is a part of x."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    g = torch.Generator(device=cuda).manual_seed(T)
    n = lambda *s: torch.randn(*s, device=cuda, generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x, w, b, st = n(5, T, C), n(C, 4), n(C), n(5, 3, C)
    y, so = ops.gdr_conv_forward(x, w, b, st)
    mine = x.clone()
    y1, so1 = ops.gdr_conv_forward(mine, w, b, st, y=mine)
    assert y1 is mine and torch.equal(y, y1) and torch.equal(so, so1)
    spans = torch.tensor([[0, T], [T, T], [2 * T, 3 * T]], dtype=torch.int32, device=cuda)
    rows = x.view(5 * T, C)
    y, so = ops.gdr_conv_forward(rows, w, b, st[:3], spans=spans, T=T, y=rows.clone())
    mine = rows.clone()
    y1, so1 = ops.gdr_conv_forward(mine, w, b, st[:3], spans=spans, T=T, y=mine)
    assert torch.equal(y, y1) and torch.equal(so, so1)
    mine = n(17, C)
    with pytest.raises(_lib.GdrError, match="overlap"):
        ops.gdr_conv_forward(mine, w, b, T=17, y=mine)


@pytest.mark.parametrize("K", [1, 4, 8])
@pytest.mark.parametrize("dtype,C", [("bf16", 264), ("f32", 33)])
def test_conv_gradient_over_its_input(cuda, dtype, C, K):
    """dx over dy, and over x, as y over x (through the C entry point, as the
    wrapper allocates dx)."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    B, T = 3, 16
    g = torch.Generator(device=cuda).manual_seed(K)
    n = lambda *s: torch.randn(*s, device=cuda, generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x, dy, w, b, st = n(B, T, C), n(B, T, C), n(C, K), n(C), n(B, K - 1, C)
    want = ops.gdr_conv_backward(x, w, b, st, dy, want_dstate=True)
    dt = _lib.GDR_BF16 if dtype == "bf16" else _lib.GDR_F32
    shape = _lib.GdrConvShape(B, T, B * T, C, K, 0, dt, dt, _lib.GDR_ACT_SILU, 0)
    size = _lib.size_of("gdr_conv_backward_workspace_bytes", shape)
    ws = torch.empty(size, dtype=torch.uint8, device=cuda)
    for over in (x, dy):
        mine = over.clone()
        ins = [mine if t is over else t for t in (x, dy)]
        dw, db, ds = torch.empty_like(w), torch.empty_like(b), torch.empty_like(st)
        ptrs = [t.data_ptr() for t in (ins[0], w, b, st)] + [0, ins[1].data_ptr(), 0]
        ptrs += [t.data_ptr() for t in (mine, dw, db, ds, ws)]
        assert _lib.layer_raw("gdr_conv_backward", shape, ptrs, torch.cuda.current_stream().cuda_stream, size) == 0
        assert same([mine, dw, db, ds], want)


def test_conv_between_its_rows(cuda):
    """A y in the gap between x's rows overlaps none of them."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    w = torch.randn(32, 4, device=cuda)
    wide = torch.randn(2, 2048, device=cuda)
    want, _ = ops.gdr_conv_forward(wide[:, :32].contiguous(), w, T=2)
    y = wide[0, 64:128].view(2, 32)
    got, _ = ops.gdr_conv_forward(wide[:, :32], w, T=2, y=y)
    assert got is y and torch.equal(got, want)


# ---- partial sums of packed rows ---------------------------------------------------

def many_spans(r, B, longest):
    """B sequences with gaps, every third of few rows, some empty ones wherever
    (0, 0) puts them, and rows behind the last."""
    at, out = int(r.integers(0, 5)), []
    for b in range(B):
        n = int(r.integers(0, 4 if b % 3 else longest))
        out.append((at, at + n) if n else (0, 0))
        at += n + int(r.integers(0, 3)) * int(r.integers(0, 40))
    return out, at + 3


def outside(rows, seqs):
    m = np.ones(rows, bool)
    for i, j in seqs:
        m[i:j] = False
    return m


def spoiled(d, seqs):
    """NaN in the rows of no sequence."""
    d[outside(len(d), seqs)] = float("nan")
    return d


def scratch(size, name, shape, device):
    """A workspace of the size that the call asks for, full of NaN."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    n = _lib.size_of(name, shape)
    assert n <= size
    return torch.full((n // 4,), float("nan"), device=device)


@pytest.mark.parametrize("dtype,C", [("bf16", 40), ("f32", 36), ("f32", 33)])
@pytest.mark.parametrize("B,longest", [(3, 700), (150, 100), (70, 300)])
def test_conv_sums_of_packed_rows(cuda, dtype, C, B, longest):
    """T not stated, so as long as all rows: dweight and dbias from the pieces
    that there are, whatever the workspace held."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    K, r = 4, np.random.default_rng(B)
    seqs, rows = many_spans(r, B, longest)
    rnd = lambda *s: torch.from_numpy(r.normal(size=s)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x, dy, w, b, st = rnd(rows, C), rnd(rows, C), rnd(C, K), rnd(C), rnd(B, K - 1, C)
    spans = torch.tensor(seqs, dtype=torch.int32, device=cuda)
    args = [spoiled(x.to(cuda), seqs), w.to(cuda), b.to(cuda), st.to(cuda), spoiled(dy.to(cuda), seqs)]
    dt = _lib.GDR_BF16 if dtype == "bf16" else _lib.GDR_F32
    shape = _lib.GdrConvShape(B, rows, rows, C, K, 0, dt, dt, _lib.GDR_ACT_SILU, 0)
    ws = scratch((rows // 64 + B) * (K + 1) * C * 4, "gdr_conv_backward_workspace_bytes", shape, cuda)
    got = ops.gdr_conv_backward(*args, spans=spans, want_dstate=True, workspace=ws)
    again = ops.gdr_conv_backward(*args, spans=spans, want_dstate=True, workspace=ws)
    assert same(got, again)
    f = lambda t: t.double().numpy()
    ref, mag = (L.conv_backward(f(x), f(w), f(b), f(st), True, seqs, f(dy), mag=m) for m in (False, True))
    check("dx", got[0], ref[0], mag[0], dtype, 64)
    check("dweight", got[1], ref[1], mag[1], dtype, 64 + rows)
    check("dbias", got[2], ref[2], mag[2], dtype, 64 + rows)
    check("dstate", got[3], ref[3], mag[3], dtype, 64)
    assert not got[0][outside(rows, seqs)].any()


@pytest.mark.parametrize("dtype,C,N,G", [("bf16", 40, 16, 1), ("f32", 70, 7, 2), ("f32", 24, 40, 1)])
@pytest.mark.parametrize("B,longest", [(3, 700), (150, 60)])
def test_scan_sums_of_packed_rows(cuda, dtype, C, N, G, B, longest):
    """The same for the scan, whose saved states and chunks ask for ascending
    sequences (an empty one may lie anywhere)."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    seqs, rows = many_spans(np.random.default_rng(B + N), B, longest)
    p = scan_inputs(dtype, B, rows, C, N, G, B)
    d = {k: dev_of(v, "f32" if k in F32 else dtype, cuda) for k, v in p.items()}
    for k in ("u", "dt", "z", "Bm", "Cm", "dy"):
        spoiled(d[k], seqs)
    spans = torch.tensor(seqs, dtype=torch.int32, device=cuda)
    y, S_T, saved = ops.gdr_scan_forward(*[d[k] for k in ARGS], spans=spans)
    dt = _lib.GDR_BF16 if dtype == "bf16" else _lib.GDR_F32
    shape = _lib.GdrScanShape(B, rows, rows, C, N, G, 0, 0, 0, 0, 0, dt, 1)
    ws = scratch(1 << 30, "gdr_scan_backward_workspace_bytes", shape, cuda)
    got = [ops.gdr_scan_backward(*[d[k] for k in ARGS[:8]], saved, d["dy"], d["dS_T"], workspace=ws)
           for _ in range(2)]
    assert same(*got)
    args = [p[k] for k in ARGS] + [True, seqs]
    n = 128 + 4 * longest
    ref, mag = (L.scan_forward(*args, mag=m) for m in (False, True))
    check("y", y, ref[0], mag[0], dtype, n)
    check("S_T", S_T, ref[1], mag[1], "f32", n)
    ref, mag = (L.scan_backward(*args, p["dy"], p["dS_T"], mag=m) for m in (False, True))
    for k, g in zip(GRADS, got[0]):
        check(k, g, ref[k], mag[k], "f32" if k in F32 else dtype,
              2 * n + (rows if k in ("dA", "dD", "ddt_bias") else 128))


# ---- the measurement hook ----------------------------------------------------------

def test_every_call_records_every_event(cuda):
    """One call at a time, over events recorded before it: the hook's events
    all move behind a mark set just before the call, in order, and a kernel's
    time lies between those of two launches."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    s = small_state(cuda)
    _, _, saved = ops.gdr_scan_forward(*s["scan"])
    _, stats = ops.gdr_norm_forward(*s["norm"], groups=4)
    calls = [  # with their kernels: 2 x 150 steps of the scan run in chunks
        (1, lambda: ops.gdr_conv_forward(*s["conv"])),
        (2, lambda: ops.gdr_conv_backward(*s["conv"], s["dy"])),
        (2, lambda: ops.gdr_scan_forward(*s["scan"])),
        (3, lambda: ops.gdr_scan_backward(*s["scan"][:8], saved, s["dy"])),
        (1, lambda: ops.gdr_norm_forward(*s["norm"], groups=4)),
        (2, lambda: ops.gdr_norm_backward(*s["norm"], stats, s["dy"], groups=4))]
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    first, mark = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    busy = torch.zeros(1 << 24, device=cuda)
    for kernels, call in calls:
        call()
        torch.cuda.synchronize()
        first.record()
        for e in events:
            e.record()
        busy.add_(1)  # (tens of microseconds between the first records and the mark)
        mark.record()
        assert _lib.set_launch_events([e.cuda_event for e in events]) == 0
        try:
            call()
        finally:
            assert _lib.set_launch_events([]) == 0
        torch.cuda.synchronize()
        start = first.elapsed_time(mark)
        times = [first.elapsed_time(e) for e in events]
        assert start > 0 and times[0] > start, (kernels, start, times)
        assert all(b > a for a, b in zip(times[:kernels], times[1:kernels])), (kernels, times)
        assert all(b >= a for a, b in zip(times, times[1:])), (kernels, times)
