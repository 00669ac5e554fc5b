"""GPU parity of the short causal convolution, the selective state space scan
and the group norm against their float64 oracle, element by element.

Tolerance.  An output element is off by at most
    half |ref| + n 2^-24 mag + 1e-30,
half a rounding step of its type (2^-8 bf16, 0 for what stays in fp32 as the
fp32 store is among the n), mag the sum of the absolute values of its terms
(the oracle's mag=True), n the roundings in fp32 on the way to it:
  * conv: K products and sums, the activation (an exponential whose argument
    |s| <= 30 carries |s| units, a reciprocal and two products): n = 64; the
    weight's gradients add one sum per row: n = 64 + rows.
  * scan: delta carries at most 3 |raw| + 8 <= 64 units (|raw| <= 18); a
    decay's argument error |delta A| (units of delta + 2) is weighted by the
    decay itself, |x| e^-|x| < 0.37 over any path, so the decays of a path
    carry at most 0.37 * 66 + 4 per step: n = 128 + 4 steps forward, twice
    that backward (the adjoint runs over the states), plus one per row in the
    sums over rows, and the 64 channels, 4 waves and tiles of a group.
  * norm: sums of up to 16 terms a lane, then a tree; the statistics' errors
    enter twice: n = 128, plus one per row in the sums over rows.
"""
import numpy as np
import pytest

import oracle.layer_oracle as L

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}


def torch_type(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def round_to(a, dtype):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch_type(dtype))
    return t.double().numpy()


def dev_of(a, dtype, dev):
    import torch
    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev).to(torch_type(dtype))


def wide(t, pad=8):
    """The same rows as a slice of wider ones (a row stride), pad elements
    before and 2 pad behind, filled with NaN."""
    import torch
    if t is None:
        return None
    lead = t.shape[:-1]
    w = torch.full((*lead, t.shape[-1] + 3 * pad), float("nan"), dtype=t.dtype, device=t.device)
    w[..., pad:pad + t.shape[-1]] = t
    return w[..., pad:pad + t.shape[-1]]


def check(name, got, ref, mag, dtype, n):
    got = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    tol = HALF[dtype] * np.abs(ref) + (n + 1) * ULP * mag * (1 + HALF[dtype]) + 1e-30
    off = np.abs(got - ref) / tol
    worst = float(off.max(initial=0.0))
    if worst > 1.0:
        pytest.fail(f"{name}: {worst:.2f} of the tolerance at {np.unravel_index(off.argmax(), off.shape)}")


def seqs_of(B, T, spans):
    return spans if spans is not None else [(b * T, (b + 1) * T) for b in range(B)]


def dev_spans(spans, dev):
    import torch
    return None if spans is None else torch.tensor(spans, dtype=torch.int32, device=dev).reshape(-1, 2)


def spoil(a, seqs):
    """NaN in the rows of no sequence: nothing may read them."""
    if a is not None:
        a[outside(len(a), seqs)] = float("nan")
    return a


def outside(rows, seqs):
    m = np.ones(rows, bool)
    for i, j in seqs:
        m[i:j] = False
    return m


# packed prompts: empty ones, one row, gaps, rows before the first and behind
# the last
PACKED = [(2, 2), (2, 3), (5, 40), (40, 40), (40, 75), (80, 81), (81, 146), (150, 150)]
PACKED_ROWS = 153


# ---- convolution ---------------------------------------------------------------

def conv_case(dev, dtype, B, T, C, K, *, wdtype=None, act="silu", bias=True, state=True, spans=None,
              rows=None, stride=False, seed=0):
    from gated_delta_rule_recurrence_amd import ops
    r = np.random.default_rng(seed)
    wdtype = wdtype or dtype
    rows = B * T if rows is None else rows
    n = lambda *s: round_to(r.normal(size=s), dtype)
    x, dy = n(rows, C), n(rows, C)
    w, b = round_to(r.normal(size=(C, K)), wdtype), round_to(r.normal(size=C), wdtype) if bias else None
    st = n(B, K - 1, C) if state else None
    dso = n(B, K - 1, C)
    seqs = seqs_of(B, T, spans)
    longest = T if spans is None else max([j - i for i, j in seqs] + [0])
    xd = spoil(dev_of(x, dtype, dev), seqs)
    xd = wide(xd) if stride else xd
    args = [xd, dev_of(w, wdtype, dev), dev_of(b, wdtype, dev), dev_of(st, dtype, dev)]
    kw = dict(act=act, spans=dev_spans(spans, dev), T=longest)
    y, so = ops.gdr_conv_forward(*args, **kw)
    dx, dw, db, ds = ops.gdr_conv_backward(*args, spoil(dev_of(dy, dtype, dev), seqs), dev_of(dso, dtype, dev),
                                           want_dstate=True, **kw)
    a = act == "silu"
    ref, mag = (L.conv_forward(x, w, b, st, a, seqs, mag=m) for m in (False, True))
    check("y", y, ref[0], mag[0], dtype, 64)
    np.testing.assert_array_equal(so.double().cpu().numpy(), ref[1])  # copies
    ref, mag = (L.conv_backward(x, w, b, st, a, seqs, dy, dso, mag=m) for m in (False, True))
    check("dx", dx, ref[0], mag[0], dtype, 64)
    check("dweight", dw, ref[1], mag[1], wdtype, 64 + rows)
    if bias:
        check("dbias", db, ref[2], mag[2], wdtype, 64 + rows)
    else:
        assert db is None
    check("dstate", ds, ref[3], mag[3], dtype, 64)
    out = outside(rows, seqs)
    assert not y.view(rows, C)[out].any() and not dx.view(rows, C)[out].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_taps(cuda, dtype, K):
    conv_case(cuda, dtype, 2, 37, 24, K, seed=K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (3, 2, 520), (1, 3, 1), (2, 17, 77), (1, 130, 33),
                                   (5, 1, 640), (1, 300, 2056), (2, 64, 512)])
def test_conv_sizes(cuda, dtype, B, T, C):
    conv_case(cuda, dtype, B, T, C, 4, seed=T)


@pytest.mark.parametrize("dtype,C", [("bf16", 40), ("f32", 30)])
def test_conv_packed(cuda, dtype, C):
    conv_case(cuda, dtype, len(PACKED), 0, C, 4, spans=PACKED, rows=PACKED_ROWS)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 8])
def test_conv_single_tokens(cuda, K):
    """One token for some of the sequences, none for the others."""
    spans = [(0, 1), (1, 1), (1, 2), (3, 4), (4, 4)]
    for dtype, C in (("bf16", 2056), ("f32", 33)):
        conv_case(cuda, dtype, 5, 0, C, K, spans=spans, rows=6, seed=K)
        conv_case(cuda, dtype, 5, 0, C, K, spans=[(2, 2)] * 5, rows=6, state=K != 3, seed=K)


@pytest.mark.parametrize("kw", [dict(bias=False), dict(state=False), dict(act="none"), dict(stride=True),
                                dict(wdtype="f32"), dict(stride=True, bias=False, state=False)])
def test_conv_options(cuda, kw):
    conv_case(cuda, "bf16", 2, 45, 48, 4, **kw)


def test_conv_odd_stride(cuda):
    """Rows that vector loads cannot take: an odd row stride of the same
    values gives the same bits."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    g = torch.Generator(device=cuda).manual_seed(1)
    x = torch.randn(2, 50, 32, device=cuda, generator=g).bfloat16()
    w = torch.randn(32, 4, device=cuda, generator=g).bfloat16()
    odd = torch.zeros(2, 50, 35, dtype=x.dtype, device=cuda)
    odd[..., :32] = x
    a, sa = ops.gdr_conv_forward(x, w)
    b, sb = ops.gdr_conv_forward(odd[..., :32], w)
    assert torch.equal(a, b) and torch.equal(sa, sb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_tokens_follow_the_prompt(cuda, dtype):
    """Prompt, then tokens one by one with the window updated in place:
    bitwise one call over all of it."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    g = torch.Generator(device=cuda).manual_seed(2)
    x = torch.randn(3, 70, 40, device=cuda, generator=g).to(torch_type(dtype))
    w, b = (torch.randn(*s, device=cuda, generator=g).to(x.dtype) for s in ((40, 4), (40,)))
    whole, end = ops.gdr_conv_forward(x, w, b)
    y, st = ops.gdr_conv_forward(x[:, :64].contiguous(), w, b)
    parts = [y]
    for t in range(64, 70):
        y, _ = ops.gdr_conv_forward(x[:, t:t + 1].contiguous(), w, b, st, state_out=st)
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, end)


# ---- scan -----------------------------------------------------------------------

def scan_inputs(dtype, B, rows, C, N, G, seed, decay=1.0):
    r = np.random.default_rng(seed)
    n = lambda *s: r.normal(size=s)
    rnd = lambda a: round_to(a, dtype)
    f32 = lambda a: round_to(a, "f32")
    step = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), C))
    return dict(u=rnd(n(rows, C)), dt=rnd(0.5 * n(rows, C)),
                A=f32(-decay * np.arange(1, N + 1) * np.exp(0.1 * n(C, N))), Bm=rnd(n(rows, G, N)),
                Cm=rnd(n(rows, G, N)), D=f32(1 + 0.1 * n(C)), z=rnd(n(rows, C)),
                dt_bias=f32(step + np.log(-np.expm1(-step))), S0=f32(0.5 * n(B, C, N)),
                dy=rnd(n(rows, C)), dS_T=f32(n(B, C, N)))


ARGS = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "S0")
GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")
F32 = {"A", "D", "dt_bias", "S0", "dS_T", "S_T", "dA", "dD", "ddt_bias", "dS0"}


def scan_case(dev, dtype, B, T, C, N, G=1, *, without=(), softplus=True, spans=None, rows=None, stride=False,
              seed=0, decay=1.0):
    from gated_delta_rule_recurrence_amd import ops
    rows = B * T if rows is None else rows
    p = scan_inputs(dtype, B, rows, C, N, G, seed, decay)
    if not softplus:
        p["dt"] = np.abs(p["dt"]) * 0.125
        p["dt_bias"] = np.abs(p["dt_bias"]) * 0.0
    for k in without:
        p[k] = None
    seqs = seqs_of(B, T, spans)
    longest = T if spans is None else max([j - i for i, j in seqs] + [0])
    d = {k: dev_of(v, "f32" if k in F32 else dtype, dev) for k, v in p.items()}
    for k in ("u", "dt", "z", "Bm", "Cm", "dy"):
        spoil(d[k], seqs)
    if stride:
        for k in ("u", "dt", "z"):
            d[k] = wide(d[k])
        for k in ("Bm", "Cm"):
            d[k] = wide(d[k].reshape(rows, G * N))
            d[k] = d[k].unflatten(-1, (G, N))
    y, S_T, saved = ops.gdr_scan_forward(*[d[k] for k in ARGS], softplus=softplus,
                                         spans=dev_spans(spans, dev), T=longest)
    y2, S2, none = ops.gdr_scan_forward(*[d[k] for k in ARGS], softplus=softplus,
                                        spans=dev_spans(spans, dev), T=longest, save=False)
    assert none is None and (y == y2).all() and (S_T == S2).all()
    grads = ops.gdr_scan_backward(*[d[k] for k in ARGS[:8]], saved, d["dy"], d["dS_T"])
    args = [p[k] for k in ARGS] + [softplus, seqs]
    ref, mag = (L.scan_forward(*args, mag=m) for m in (False, True))
    n = 128 + 4 * longest
    check("y", y, ref[0], mag[0], dtype, n)
    check("S_T", S_T, ref[1], mag[1], "f32", n)
    ref, mag = (L.scan_backward(*args, p["dy"], p["dS_T"], mag=m) for m in (False, True))
    given = dict(zip(GRADS, ARGS))
    for k, g in zip(GRADS, grads):
        if k != "dS0" and given[k] in without:
            assert g is None
            continue
        check(k, g, ref[k], mag[k], "f32" if k in F32 else dtype,
              2 * n + (rows if k in ("dA", "dD", "ddt_bias") else 128))
    out = outside(rows, seqs)
    for k, g in zip(("y",) + GRADS, (y,) + grads):
        if g is not None and k in ("y", "du", "ddt", "dB", "dC", "dz"):
            assert not g.reshape(rows, -1)[out].any(), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 4, 7, 8, 12, 16, 24, 32, 45, 64])
def test_scan_states(cuda, dtype, N):
    scan_case(cuda, dtype, 2, 37, 20, N, seed=N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,G", [(1, 1, 8, 1), (3, 2, 65, 1), (1, 15, 64, 2), (2, 16, 66, 3), (1, 17, 130, 1),
                                     (4, 1, 200, 4), (1, 64, 1, 1), (1, 65, 96, 1), (2, 300, 70, 2)])
def test_scan_sizes(cuda, dtype, B, T, C, G):
    scan_case(cuda, dtype, B, T, C, 16, G, seed=T)


# up to 4 steps (a kernel of its own), and across its border
@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("f32", 7), ("bf16", 33)])
@pytest.mark.parametrize("T", [2, 3, 4, 5])
def test_scan_few_steps(cuda, dtype, N, T):
    scan_case(cuda, dtype, 3, T, 70, N, 2, seed=T)
    scan_case(cuda, dtype, 4, 0, 35, N, spans=[(0, 1), (1, 1), (1, 1 + T), (2 + T, 3 + T)], rows=4 + T)


def test_scan_unsplit(cuda):
    """Enough waves that forward and backward run every sequence as one chunk
    of several tiles (17 x 33 channel tiles x 4 waves), in groups that end
    inside a channel tile."""
    scan_case(cuda, "f32", 17, 35, 2112, 4, 1)
    scan_case(cuda, "bf16", 19, 21, 2100, 3, 4)


@pytest.mark.parametrize("T,C,N", [(1000, 24, 16), (2100, 8, 5), (700, 16, 40)])
def test_scan_many_chunks(cuda, T, C, N):
    """Sequences split into up to 64 chunks; a batch of unequal ones too."""
    scan_case(cuda, "f32", 1, T, C, N, seed=T)
    scan_case(cuda, "f32", 3, 0, C, N, spans=[(0, T // 3), (T // 3, T // 3 + 1), (T // 2, T)], rows=T + 5)


@pytest.mark.parametrize("dtype,N", [("bf16", 16), ("f32", 10), ("f32", 40)])
def test_scan_packed(cuda, dtype, N):
    scan_case(cuda, dtype, len(PACKED), 0, 40, N, 2, spans=PACKED, rows=PACKED_ROWS)


@pytest.mark.parametrize("kw", [dict(without=("D",)), dict(without=("z",)), dict(without=("dt_bias",)),
                                dict(without=("S0", "dS_T")), dict(softplus=False), dict(stride=True),
                                dict(without=("D", "z", "dt_bias", "S0", "dS_T"), softplus=False),
                                dict(decay=40.0), dict(decay=1e-3)])
def test_scan_options(cuda, kw):
    scan_case(cuda, "f32", 2, 100, 48, 16, 2, **kw)
    scan_case(cuda, "bf16", 1, 33, 48, 16, 1, **kw)


def test_scan_tokens_follow_the_prompt(cuda):
    """Prompt, then tokens one by one with the state updated in place, against
    one call over all of it: the recurrence is the same, only the prompt's
    split into chunks rounds differently."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    B, T, C, N = 2, 90, 72, 16
    p = scan_inputs("f32", B, B * T, C, N, 1, 4)
    d = {k: dev_of(v, "f32", cuda) for k, v in p.items()}
    for k in ("u", "dt", "z", "Bm", "Cm"):
        d[k] = d[k].reshape(B, T, *d[k].shape[1:])
    call = lambda a, b, S0, **kw: ops.gdr_scan_forward(
        *[d[k][:, a:b].contiguous() if k in ("u", "dt", "z", "Bm", "Cm") else d[k] for k in ARGS[:8]], S0,
        save=False, **kw)
    whole, end, _ = call(0, T, d["S0"])
    y, S, _ = call(0, 80, d["S0"])
    parts = [y]
    for t in range(80, T):
        y, _, _ = call(t, t + 1, S, S_T=S)
        parts.append(y)
    mag = L.scan_forward(*[p[k] for k in ARGS], True, seqs_of(B, T, None), mag=True)
    check("y", torch.cat(parts, 1), whole.double().cpu().numpy(), mag[0].reshape(B, T, C), "f32", 2 * (128 + 4 * T))
    check("S_T", S, end.double().cpu().numpy(), mag[1], "f32", 2 * (128 + 4 * T))


# ---- norm -----------------------------------------------------------------------

def norm_case(dev, dtype, rows, C, G, *, wdtype=None, center=False, act="silu", gate=True, weight=True, bias=True,
              shared=False, stride=False, seed=0, shift=0.0):
    from gated_delta_rule_recurrence_amd import ops
    r = np.random.default_rng(seed)
    wdtype = wdtype or dtype
    n = lambda *s: round_to(r.normal(size=s), dtype)
    x, dy, z = round_to(r.normal(size=(rows, C)) + shift, dtype), n(rows, C), n(rows, C) if gate else None
    width = C // G if shared else C
    w = round_to(r.normal(size=width), wdtype) if weight else None
    b = round_to(r.normal(size=width), wdtype) if bias else None
    eps = 1e-5
    xd, zd = dev_of(x, dtype, dev), dev_of(z, dtype, dev)
    if stride:
        xd, zd = wide(xd), wide(zd, 16)
    args = [xd, dev_of(w, wdtype, dev), dev_of(b, wdtype, dev), zd]
    kw = dict(groups=G, center=center, act=act)
    y, stats = ops.gdr_norm_forward(*args, eps=eps, **kw)
    dx, dw, db, dz = ops.gdr_norm_backward(*args, stats, dev_of(dy, dtype, dev), **kw)
    eps = float(np.float32(eps))
    a = act == "silu"
    ref, mag = (L.norm_forward(x, w, b, z, G, eps, center, a, mag=m) for m in (False, True))
    check("y", y, ref, mag, dtype, 128)
    ref, mag = (L.norm_backward(x, w, b, z, G, eps, center, a, dy, mag=m) for m in (False, True))
    fold = (lambda g: g.reshape(G, -1).sum(0)) if shared else (lambda g: g)
    check("dx", dx, ref[0], mag[0], dtype, 128)
    for name, g, have, i in (("dweight", dw, weight, 1), ("dbias", db, bias, 2)):
        if have:
            check(name, g, fold(ref[i]), fold(mag[i]), wdtype, 128 + rows * (G if shared else 1))
        else:
            assert g is None
    if gate:
        check("dz", dz, ref[3], mag[3], dtype, 128)
    else:
        assert dz is None


# every lane count and vector count of the kernels, whole and ragged
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 5, 8, 24, 64, 72, 128, 100, 200, 256, 333, 512, 520, 700, 1024, 1500, 2048,
                               2052, 4096, 4500, 8192])
def test_norm_widths(cuda, dtype, D):
    norm_case(cuda, dtype, 3, 2 * D, 2, center=D % 2 == 0, seed=D)


@pytest.mark.parametrize("rows,G", [(1, 1), (2, 3), (7, 5), (100, 12), (33, 64), (517, 6)])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_rows(cuda, rows, G, shared):
    norm_case(cuda, "f32", rows, G * 40, G, shared=shared, seed=rows)
    norm_case(cuda, "bf16", rows, G * 128, G, shared=shared, center=True, seed=rows)


@pytest.mark.parametrize("kw", [dict(gate=False), dict(act="none"), dict(gate=False, act="none"), dict(weight=False),
                                dict(bias=False), dict(weight=False, bias=False), dict(center=True, gate=False),
                                dict(center=True, shift=3.0), dict(stride=True), dict(wdtype="f32"),
                                dict(stride=True, shared=True, center=True)])
def test_norm_options(cuda, kw):
    norm_case(cuda, "bf16", 19, 192, 3, **kw)
    norm_case(cuda, "f32", 19, 192, 3, **{**kw, "wdtype": "bf16" if "wdtype" in kw else None})


@pytest.mark.parametrize("dtype,rows,C,G,shared", [("f32", 60000, 8, 1, False), ("bf16", 30000, 24, 2, True),
                                                   ("f32", 1300, 1500, 1, False), ("bf16", 1300, 6000, 2, True)])
def test_norm_many_rows(cuda, dtype, rows, C, G, shared):
    """More rows than the walkers of the grid take in one turn."""
    norm_case(cuda, dtype, rows, C, G, shared=shared, center=shared, seed=rows)


def some_spans(r, B):
    """B ascending spans with gaps, some empty, and rows behind the last."""
    at = np.sort(r.integers(0, 160, size=2 * B))
    return [(int(at[2 * b]), int(at[2 * b + 1])) for b in range(B)], int(at[-1]) + int(r.integers(0, 5))


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(cuda, seed):
    r = np.random.default_rng(1000 + seed)
    pick = lambda *v: v[int(r.integers(len(v)))]
    flip = lambda: bool(r.integers(2))
    dtype, B, T = pick("bf16", "f32"), int(r.integers(1, 6)), int(r.integers(1, 120))
    spans, rows = some_spans(r, B) if flip() else (None, None)
    G = int(r.integers(1, 4))
    C, N, K = G * int(r.integers(1, 90)), int(r.integers(1, 65)), int(r.integers(1, 9))
    case = dict(dtype=dtype, B=B, T=T, spans=spans, rows=rows, C=C, G=G, N=N, K=K)
    print(case, flush=True)
    conv_case(cuda, dtype, B, T, C, K, wdtype=pick(None, "f32", "bf16"), act=pick("silu", "none"), bias=flip(),
              state=flip(), spans=spans, rows=rows, stride=flip(), seed=seed)
    without = [k for k in ("D", "z", "dt_bias", "S0", "dS_T") if flip()]
    scan_case(cuda, dtype, B, T, C, N, G, without=without, spans=spans, rows=rows, stride=flip(), seed=seed)
    norm_case(cuda, dtype, int(r.integers(1, 400)), C, G, wdtype=pick(None, "f32", "bf16"), center=flip(),
              act=pick("silu", "none"), gate=flip(), weight=flip(), bias=flip(), shared=flip(), stride=flip(),
              seed=seed)


# ---- all three: streams, graphs, repeats, spans, large offsets ----------------------

def small_state(dev, dtype="bf16", seed=0):
    """Inputs of one small call of each operator."""
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s: torch.randn(*s, device=dev, generator=g)
    t = torch_type(dtype)
    B, T, C, N = 2, 150, 96, 16
    r = lambda *s: n(*s).to(t)
    return dict(conv=(r(B, T, C), r(C, 4), r(C), r(B, 3, C)), dy=r(B, T, C),
                scan=(r(B, T, C), r(B, T, C), -torch.exp(n(C, N)), r(B, T, 2, N), r(B, T, 2, N), n(C), r(B, T, C),
                      n(C), n(B, C, N)),
                norm=(r(B, T, C), r(C), r(C), r(B, T, C)))


def run_all(s):
    """Forward and backward of the three; every output, in order."""
    from gated_delta_rule_recurrence_amd import ops
    out = [*ops.gdr_conv_forward(*s["conv"])]
    out += ops.gdr_conv_backward(*s["conv"], s["dy"], want_dstate=True)
    y, S_T, saved = ops.gdr_scan_forward(*s["scan"])
    out += [y, S_T, *ops.gdr_scan_backward(*s["scan"][:8], saved, s["dy"])]
    y, stats = ops.gdr_norm_forward(*s["norm"], groups=4, center=True)
    out += [y, *ops.gdr_norm_backward(*s["norm"], stats, s["dy"], groups=4, center=True)]
    return out


def same(a, b):
    import torch
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_are_bitwise_equal(cuda, dtype):
    s = small_state(cuda, dtype)
    first = run_all(s)
    for _ in range(3):
        assert same(run_all(s), first)


def test_another_stream(cuda):
    import torch
    s = small_state(cuda)
    first = run_all(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run_all(s)
    torch.cuda.current_stream().wait_stream(side)
    assert same(out, first)


def test_two_streams_at_once(cuda):
    """Two calls in flight share no library state."""
    import torch
    states = [small_state(cuda, seed=k) for k in range(2)]
    want = [run_all(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for _ in range(5):
        got = []
        for st, s in zip(streams, states):
            with torch.cuda.stream(st):
                got.append(run_all(s))
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_captured_and_replayed(cuda):
    """A graph of all forward and backward calls, replayed on new inputs with
    eager calls and synchronizations between."""
    import torch
    s = small_state(cuda)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_all(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_all(s)
    flat = lambda d: [t for k in ("conv", "scan", "norm") for t in d[k]] + [d["dy"]]
    for seed in (1, 2, 3):
        new = small_state(cuda, seed=seed)
        for a, b in zip(flat(s), flat(new)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, run_all(new)), seed
        graph.replay()
        assert same(out, run_all(s)), seed


def run_packed(s, spans, T, window=None, states=None):
    """Forward and backward of the convolution and the scan over packed rows;
    states in place where they are given."""
    from gated_delta_rule_recurrence_amd import ops
    flat = lambda t: None if t is None else t.reshape(-1, *t.shape[2:])
    x, w, b, _ = s["conv"]
    kw = dict(spans=spans, T=T)
    y, win = ops.gdr_conv_forward(flat(x), w, b, window, state_out=window, **kw)
    out = [y, win, *ops.gdr_conv_backward(flat(x), w, b, None, flat(s["dy"]), **kw)[:3]]
    u, dt, A, Bm, Cm, D, z, bias, _ = s["scan"]
    args = flat(u), flat(dt), A, flat(Bm), flat(Cm), D, flat(z), bias
    y, S_T, saved = ops.gdr_scan_forward(*args, states, S_T=states, **kw)
    return out + [y, S_T, *ops.gdr_scan_backward(*args, saved, flat(s["dy"]), want_dS0=False)[:8]]


def test_a_graph_whose_spans_change(cuda):
    """A graph over packed rows, replayed on other cuts of the rows (empty
    sequences, gaps, one long one), its states carried from replay to replay."""
    import torch
    s = small_state(cuda, seed=4)
    cuts = [[(0, 100), (100, 100), (110, 290)], [(0, 0), (3, 4), (4, 300)], [(290, 300), (300, 300), (300, 300)],
            [(0, 20), (40, 60), (80, 297)]]
    spans = torch.tensor(cuts[0], dtype=torch.int32, device=cuda)
    window, S = torch.zeros(3, 3, 96, dtype=torch.bfloat16, device=cuda), torch.zeros(3, 96, 16, device=cuda)
    mine, mine_S = window.clone(), S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_packed(s, spans, 300, window, S)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_packed(s, spans, 300, window, S)
    window.zero_(), S.zero_()
    for cut in cuts:
        spans.copy_(torch.tensor(cut, dtype=torch.int32, device=cuda))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, run_packed(s, spans, 300, mine, mine_S)), cut
        assert torch.equal(window, mine) and torch.equal(S, mine_S)


def test_states_in_place(cuda):
    """state_out = state and S_T = S0, over prompts of several tiles and
    chunks: the values of the call with buffers apart."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda)
    x, w, b, st = s["conv"]
    y0, so = ops.gdr_conv_forward(x, w, b, st)
    mine = st.clone()
    y1, _ = ops.gdr_conv_forward(x, w, b, mine, state_out=mine)
    assert torch.equal(y0, y1) and torch.equal(so, mine)
    y0, S_T, _ = ops.gdr_scan_forward(*s["scan"], save=False)
    mine = s["scan"][8].clone()
    y1, _, _ = ops.gdr_scan_forward(*s["scan"][:8], mine, save=False, S_T=mine)
    assert torch.equal(y0, y1) and torch.equal(S_T, mine)
    x, w, b, z = s["norm"]
    y0, _ = ops.gdr_norm_forward(x, w, b, z, groups=4)
    mine = x.clone()
    ops.gdr_norm_forward(mine, w, b, z, groups=4, y=mine)
    assert torch.equal(y0, mine)


def test_split_scan_in_place(cuda):
    """S_T = S0 where many workgroups share a sequence's chunks, more than the
    device holds at once: packed sequences of many chunks, one and none."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    g = torch.Generator(device=cuda).manual_seed(5)
    C, N, rows = 4096, 16, 6144
    spans = torch.tensor([[0, 4000], [4000, 4000], [4000, 4020], [4020, rows]], dtype=torch.int32,
                         device=cuda)

    def rand(*shape):
        return torch.randn(*shape, device=cuda, generator=g)

    u, dt = rand(rows, C).bfloat16(), rand(rows, C).bfloat16()
    A, S0 = -torch.exp(rand(C, N)), rand(4, C, N)
    Bm, Cm = rand(rows, 1, N).bfloat16(), rand(rows, 1, N).bfloat16()
    y0, S_T, _ = ops.gdr_scan_forward(u, dt, A, Bm, Cm, S0=S0, spans=spans, T=4000, save=False)
    for _ in range(4):
        mine = S0.clone()
        y1, _, _ = ops.gdr_scan_forward(u, dt, A, Bm, Cm, S0=mine, spans=spans, T=4000, save=False,
                                        S_T=mine)
        assert torch.equal(y0, y1) and torch.equal(S_T, mine)


def test_spans_are_cut_to_the_rows(cuda):
    """Spans outside 0 .. rows, and longer than T."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda)
    rows = lambda t: t.reshape(300, *t.shape[2:])
    wild = torch.tensor([[-7, 100], [100, 90], [120, 150], [200, 1 << 30]], dtype=torch.int32, device=cuda)
    tame = torch.tensor([[0, 80], [100, 100], [120, 150], [200, 280]], dtype=torch.int32, device=cuda)
    got = []
    for spans in (wild, tame):
        x, w, b, st = s["conv"]
        st = torch.cat([st, st])
        out = [*ops.gdr_conv_forward(rows(x), w, b, st, spans=spans, T=80)]
        out += ops.gdr_conv_backward(rows(x), w, b, st, rows(s["dy"]), spans=spans, T=80, want_dstate=True)
        u, dt, A, Bm, Cm, D, z, bias, S0 = s["scan"]
        args = [rows(u), rows(dt), A, rows(Bm), rows(Cm), D, rows(z), bias]
        y, S_T, saved = ops.gdr_scan_forward(*args, torch.cat([S0, S0]), spans=spans, T=80)
        out += [y, S_T, *ops.gdr_scan_backward(*args, saved, rows(s["dy"]))]
        got.append(out)
    assert same(*got)


def test_a_longest_length_far_above_the_rows(cuda):
    """T is a bound: grids that follow it are cut to what a launch takes."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda)
    spans = torch.tensor([[0, 80], [100, 290]], dtype=torch.int32, device=cuda)

    def rows(t):
        return t.reshape(300, *t.shape[2:])[..., :8].contiguous()

    x, w, b, st = s["conv"]
    x, dy, w, b, st = rows(x), rows(s["dy"]), w[:8].contiguous(), b[:8].contiguous(), st[..., :8].contiguous()
    u, dt, A, Bm, Cm, D, z, bias, S0 = s["scan"]
    u, dt, z, A, D, bias, S0 = (rows(u), rows(dt), rows(z), A[:8].contiguous(), D[:8].contiguous(),
                                bias[:8].contiguous(), S0[:, :8].contiguous())
    Bm, Cm = Bm.reshape(300, *Bm.shape[2:])[:, :1].contiguous(), Cm.reshape(300, *Cm.shape[2:])[:, :1].contiguous()
    args = u, dt, A, Bm, Cm, D, z, bias
    got = []
    for T in (190, 2 ** 30 - 1):
        out = [*ops.gdr_conv_forward(x, w, b, st, spans=spans, T=T)]
        out += ops.gdr_conv_backward(x, w, b, st, dy, spans=spans, T=T, want_dstate=True)
        y, S_T, saved = ops.gdr_scan_forward(*args, S0, spans=spans, T=T)
        out += [y, S_T, *ops.gdr_scan_backward(*args, saved, dy)]
        got.append(out)
    # Other tiles and chunks, so other orders of the same sums: each side within
    # 128 + 4 * 190 + 300 < 1200 roundings of 2^-24 of the sum of magnitudes, taken as
    # at most 7 times the largest value of the tensor (1e-3 = 2400 * 7 * 2^-24), and a
    # rounded bf16 within a whole step, 2^-7.
    for a, b in zip(*got):
        a, b = a.float(), b.float()
        assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-3 * a.abs().max()).all()


@pytest.mark.parametrize("T", [1, 20])
def test_steps_keep_their_relative_accuracy(cuda, T):
    """y = delta where u, B and C are 1 and nothing is carried (A so low that
    every decay is 0): softplus over its range, tiny steps included.  The
    exponential's argument is rounded twice, |raw| units each, and the constant
    in it once more; then come fewer than 8 roundings, with the logarithm's."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    C = 4096
    raw = np.linspace(-86.0, 90.0, T * C).astype(np.float32)
    dt = torch.from_numpy(raw).to(cuda).view(1, T, C)
    one = torch.ones(1, T, 1, 1, device=cuda)
    A = torch.full((C, 1), -float("inf"), device=cuda)
    y, _, _ = ops.gdr_scan_forward(torch.ones_like(dt), dt, A, one, one, save=False)
    x = raw.astype(np.float64)
    ref = np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))
    off = np.abs(y.double().cpu().numpy().ravel() - ref) / ref
    assert (off <= (3 * np.abs(np.minimum(x, 0)) + 8) * ULP).all()


def test_infinite_rates(cuda):
    """A = -inf forgets at every step, and is no matter behind a sequence's
    last step, whatever the tiles and chunks."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    for T in (1, 3, 21, 150):
        u, dt, A, Bm, Cm, D, z, bias, S0 = small_state(cuda)["scan"]
        rows = [t[:, :T].contiguous() for t in (u, dt, Bm, Cm, z)]
        got = []
        for rate in (-float("inf"), -1e30):
            A = A.clone()
            A[::3] = rate
            y, S_T, _ = ops.gdr_scan_forward(rows[0], rows[1], A, rows[2], rows[3], D, rows[4], bias, S0)
            assert torch.isfinite(y).all() and torch.isfinite(S_T).all()
            got.append((y, S_T))
        assert same(*got), T


def test_gradients_that_arrive_as_views(cuda):
    """Dense views that start off a 16-byte boundary, and sums' broadcasts."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    g = torch.Generator(device=cuda).manual_seed(11)

    def rand(*shape):
        return torch.randn(*shape, device=cuda, generator=g)

    x, w, A = rand(1, 7, 5), rand(5, 4), -torch.exp(rand(5, 3))
    Bm = rand(1, 7, 1, 3)
    dy = rand(1, 1 + 7 * 5)
    view = dy[:, 1:].view(1, 7, 5)
    assert view.is_contiguous() and view.data_ptr() % 16
    for f in (lambda t: ops.causal_conv(t, w)[0], lambda t: ops.selective_scan(t, t, A, Bm, Bm)[0],
              lambda t: ops.group_norm(t, groups=5, center=False)):
        got = []
        for d in (view, view.clone()):
            t = x.clone().requires_grad_()
            f(t).backward(d)
            got.append((t.grad,))
        assert same(*got)
        t, r = x.clone().requires_grad_(), x.clone().requires_grad_()
        f(t).sum().backward()
        f(r).backward(torch.ones_like(x))
        assert torch.equal(t.grad, r.grad)


def test_spans_changed_before_the_backward(cuda):
    import torch
    from gated_delta_rule_recurrence_amd import ops
    x = torch.randn(12, 8, device=cuda, requires_grad=True)
    A, Bm = -torch.ones(8, 4, device=cuda), torch.randn(12, 1, 4, device=cuda)
    spans = torch.tensor([[0, 12]], dtype=torch.int32, device=cuda)
    for f in (lambda: ops.causal_conv(x, torch.ones(8, 4, device=cuda), spans=spans)[0],
              lambda: ops.selective_scan(x, x, A, Bm, Bm, spans=spans)[0]):
        y = f()
        spans[0, 1] = 9
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        spans[0, 1] = 12


def test_no_rows_and_no_sequences(cuda):
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda)
    x, w, b, st = s["conv"]
    y, so = ops.gdr_conv_forward(x[:, :0], w, b, st)
    assert y.shape == (2, 0, 96) and torch.equal(so, st)
    dx, dw, db, ds = ops.gdr_conv_backward(x[:, :0], w, b, st, x[:, :0].contiguous(), st, want_dstate=True)
    assert not dw.any() and not db.any() and torch.equal(ds, st)
    u, dt, A, Bm, Cm, D, z, bias, S0 = s["scan"]
    none = [u[:, :0], dt[:, :0], A, Bm[:, :0], Cm[:, :0], D, z[:, :0], bias]
    y, S_T, saved = ops.gdr_scan_forward(*none, S0)
    assert y.shape == (2, 0, 96) and torch.equal(S_T, S0)
    g = ops.gdr_scan_backward(*none, saved, u[:, :0].contiguous(), S0)
    assert not g[2].any() and not g[5].any() and not g[7].any() and torch.equal(g[8], S0)
    none = [t[:0] if t.dim() > 2 else t for t in s["scan"]]
    y, S_T, saved = ops.gdr_scan_forward(*none)
    g = ops.gdr_scan_backward(*none[:8], saved, u[:0])
    assert y.shape == (0, 150, 96) and S_T.shape == (0, 96, 16) and not g[2].any()
    dx, dw, db, ds = ops.gdr_conv_backward(x[:0], w, b, st[:0], x[:0], want_dstate=True)
    assert not dw.any() and not db.any()
    x, w, b, z = s["norm"]
    y, stats = ops.gdr_norm_forward(x[:0], w, b, z[:0], groups=4)
    dx, dw, db, dz = ops.gdr_norm_backward(x[:0], w, b, z[:0], stats, x[:0], groups=4)
    assert y.shape == (0, 150, 96) and not dw.any() and not db.any()


def test_offsets_beyond_32_bits(cuda):
    """Rows whose elements lie past 2^32 (and states, of the norm's row count,
    past 2^31): the last sequence of a long packed buffer, against the same
    rows in a buffer of their own."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    C, R, n, N = 16384, 1 << 18, 90, 4
    g = torch.Generator(device=cuda).manual_seed(3)
    big = torch.empty(R + n, C, dtype=torch.bfloat16, device=cuda)
    tail = torch.randn(n, C, device=cuda, generator=g).bfloat16()
    big[R:] = tail
    spans = torch.tensor([[5, 40], [R, R + n]], dtype=torch.int32, device=cuda)
    big[5:40] = tail[:35]
    own = torch.tensor([[0, 35], [35, 35 + n]], dtype=torch.int32, device=cuda)
    both = torch.cat([tail[:35], tail])
    w = torch.randn(C, 4, device=cuda, generator=g).bfloat16()
    out = torch.empty_like(big)
    ops.gdr_conv_forward(big, w, spans=spans, T=n, y=out)
    y, _ = ops.gdr_conv_forward(both, w, spans=own, T=n)
    assert torch.equal(out[R:], y[35:]) and torch.equal(out[5:40], y[:35])
    A = -torch.exp(torch.randn(C, N, device=cuda, generator=g))
    bm = torch.zeros(R + n, 1, N, dtype=torch.bfloat16, device=cuda)
    mine = torch.randn(35 + n, 1, N, device=cuda, generator=g).bfloat16()
    bm[5:40], bm[R:] = mine[:35], mine[35:]
    _, S_T, _ = ops.gdr_scan_forward(big, big, A, bm, bm, spans=spans, T=n, save=False, y=out)
    y, S, _ = ops.gdr_scan_forward(both, both, A, mine, mine, spans=own, T=n, save=False)
    # (split into other chunks, so rounded otherwise)
    assert torch.allclose(S_T, S, rtol=1e-4, atol=1e-4)
    assert torch.allclose(out[R:].float(), y[35:].float(), rtol=2e-2, atol=2e-2)
    assert torch.allclose(out[5:40].float(), y[:35].float(), rtol=2e-2, atol=2e-2)
    ops.gdr_norm_forward(big, groups=128, save=False, y=out, act=None)
    y, _ = ops.gdr_norm_forward(tail, groups=128, save=False, act=None)
    assert torch.equal(out[R:], y)


def test_gradients_against_differences(cuda):
    """Central differences of the fp32 forward along a random direction v
    against the gradient.  (f(x + h v) - f(x - h v)) / 2h is the mean of
    g(e) = <grad f(x + e v), v> over [-h, h]; Simpson's rule gives that mean as
    (g(-h) + 4 g(0) + g(h)) / 6 up to h^4 / 180 of f's fifth derivative, where
    g(0) alone would leave h^2 / 6 of the third (seen in A, whose decays
    compound over 150 steps).  At h = 1e-2 that leaves the rounding of the
    difference, 2^-24 |<dy, y>|_1 / h: below 2e-3 of sum |grad v|."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda, "f32", seed=9)
    gen = torch.Generator(device=cuda).manual_seed(10)
    fs = dict(conv=lambda *a: ops.causal_conv(*a)[0], scan=lambda *a: ops.selective_scan(*a)[0],
              norm=lambda *a: ops.group_norm(*a, groups=4, center=True))
    dy, h = s["dy"], 1e-2
    for name, f in fs.items():
        args = [(t * 0.5 if name == "scan" and i != 2 else t).clone() for i, t in enumerate(s[name])]
        for i, t in enumerate(args):
            v = torch.randn(t.shape, device=cuda, generator=gen)
            value, slope, scale = {}, {}, 0.0
            for e in (-h, 0.0, h):
                x = (t + e * v).requires_grad_()
                y = f(*[x if k == i else a for k, a in enumerate(args)])
                value[e] = (y.detach().double() * dy.double()).sum()
                y.backward(dy)
                slope[e] = (x.grad.double() * v.double()).sum()
                scale = max(scale, float((x.grad.double() * v.double()).abs().sum()))
            got = (value[h] - value[-h]) / (2 * h)
            want = (slope[-h] + 4 * slope[0.0] + slope[h]) / 6
            assert abs(got - want) <= 2e-3 * scale, (name, i, float(got), float(want), scale)


def test_autograd_of_shared_and_broadcast_inputs(cuda):
    """One tensor as several inputs (its gradients add up), an expanded bias
    and a strided slice as x."""
    import torch
    from gated_delta_rule_recurrence_amd import ops
    s = small_state(cuda, "f32")
    u, dt, A, Bm, Cm, D, z, bias, S0 = s["scan"]
    one = Bm.clone().requires_grad_()
    y, _ = ops.selective_scan(u, dt, A, one, one, D, z, bias)
    y.backward(s["dy"])
    b, c = Bm.clone().requires_grad_(), Bm.clone().requires_grad_()
    y, _ = ops.selective_scan(u, dt, A, b, c, D, z, bias)
    y.backward(s["dy"])
    torch.testing.assert_close(one.grad, b.grad + c.grad, rtol=1e-6, atol=1e-6)
    x = torch.randn(2, 150, 300, device=cuda).requires_grad_()
    w = s["conv"][1]
    y, _ = ops.causal_conv(x[..., 104:200], w)
    y.backward(s["dy"])
    x2 = x.detach()[..., 104:200].contiguous().requires_grad_()
    y, _ = ops.causal_conv(x2, w)
    y.backward(s["dy"])
    assert torch.equal(x.grad[..., 104:200], x2.grad) and not x.grad[..., :104].any()


def test_refusals(cuda):
    import torch
    from gated_delta_rule_recurrence_amd import _lib, ops
    s = small_state(cuda)
    x, w, b, st = s["conv"]
    u, dt, A, Bm, Cm, D, z, bias, S0 = s["scan"]
    with pytest.raises(_lib.GdrError, match="aligned"):
        ops.gdr_conv_forward(x[..., 1:95], w[1:95].contiguous())
    with pytest.raises(_lib.GdrError, match="dimension"):
        ops.gdr_conv_forward(x, torch.zeros(96, 9, device=cuda, dtype=x.dtype))
    for bad in (lambda: ops.gdr_conv_forward(x, w.float(), b), lambda: ops.gdr_conv_forward(x, w, b, st[:1]),
                lambda: ops.gdr_conv_forward(x.half(), w), lambda: ops.gdr_conv_forward(x, w, act="tanh"),
                lambda: ops.gdr_conv_forward(x, w[:90]), lambda: ops.gdr_conv_forward(x.transpose(0, 1), w),
                lambda: ops.gdr_conv_forward(x, w, spans=torch.zeros(2, 2, device=cuda)),
                lambda: ops.gdr_conv_forward(x, w, y=torch.empty(2, 150, 95, device=cuda, dtype=x.dtype)),
                lambda: ops.gdr_scan_forward(u, dt[:, :149], A, Bm, Cm),
                lambda: ops.gdr_scan_forward(u, dt, A, Bm, Cm[:, :, :1]),
                lambda: ops.gdr_scan_forward(u, dt, A.bfloat16(), Bm, Cm),
                lambda: ops.gdr_scan_forward(u, dt.float(), A, Bm, Cm),
                lambda: ops.gdr_scan_forward(u, dt, A, Bm, Cm, S0=S0[:1]),
                lambda: ops.gdr_scan_forward(u, dt, A, Bm, Cm, z=z.cpu()),
                lambda: ops.gdr_norm_forward(x, groups=7), lambda: ops.gdr_norm_forward(x, w, groups=4),
                lambda: ops.gdr_norm_forward(x, x[0, 0, :10].contiguous(), groups=4),
                lambda: ops.gdr_norm_forward(x, z=x[:1], groups=4)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(_lib.GdrError, match="dimension"):
        ops.gdr_scan_forward(u, dt, torch.zeros(96, 65, device=cuda), torch.zeros(2, 150, 2, 65, device=cuda).bfloat16(),
                             torch.zeros(2, 150, 2, 65, device=cuda).bfloat16())
    with pytest.raises(_lib.GdrError, match="dimension"):  # groups of 3 of 96 channels: 32 a group
        ops.gdr_scan_forward(u, dt, A, Bm[:, :, :1].expand(2, 150, 5, 16).contiguous(),
                             Cm[:, :, :1].expand(2, 150, 5, 16).contiguous())
    with pytest.raises(_lib.GdrError, match="eps"):
        ops.gdr_norm_forward(x, groups=4, eps=-1.0)
    with pytest.raises(_lib.GdrError, match="dimension"):
        ops.gdr_norm_forward(torch.zeros(1, 8200, device=cuda), groups=1)


def test_launch_events_cover_the_new_calls(cuda):
    """The measurement hook: each event recorded once per call."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    s = small_state(cuda)
    want = run_all(s)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    for e in events:
        e.record()
    torch.cuda.synchronize()
    assert _lib.set_launch_events([e.cuda_event for e in events]) == 0
    try:
        got = run_all(s)
        torch.cuda.synchronize()
        spans = [a.elapsed_time(b) for a, b in zip(events, events[1:])]
    finally:
        assert _lib.set_launch_events([]) == 0
    assert same(got, want) and all(t >= 0 for t in spans)


# ---- the layer: together, through autograd ---------------------------------------

def test_layer_together(cuda):
    """q, k, v from the convolution, the recurrence, the gated norm, and the
    scan on the result: one training step through autograd against the
    composed oracles, and the same tokens served one by one."""
    import torch

    import oracle.gdr_oracle as O
    from gated_delta_rule_recurrence_amd import ops
    B, T, Hk, Hv, Dk, Dv = 2, 40, 2, 4, 16, 24
    nq, nv = Hk * Dk, Hv * Dv
    C = 2 * nq + nv
    r = np.random.default_rng(11)
    f = lambda a: round_to(a, "f32")
    x, w, b = f(r.normal(size=(B, T, C)) * 0.5), f(r.normal(size=(C, 4)) * 0.5), f(r.normal(size=C) * 0.1)
    g, beta = f(r.uniform(0.7, 1.0, (B, T, Hv))), f(r.uniform(0.2, 0.9, (B, T, Hv)))
    z, nw = f(r.normal(size=(B, T, nv))), f(1 + 0.1 * r.normal(size=Dv))
    s = scan_inputs("f32", B, B * T, nv, 8, 2, 12)
    dy = f(r.normal(size=(B, T, nv)))
    leaf = lambda a: dev_of(a, "f32", cuda).requires_grad_()
    X, W, Bi, G_, BE, Z, NW = map(leaf, (x, w, b, g, beta, z, nw))
    SC = {k: leaf(s[k]) for k in ("dt", "A", "Bm", "Cm", "D", "z", "dt_bias")}
    rows = lambda t, i=0, j=T: t.reshape(B, T, *t.shape[1:])[:, i:j].contiguous()

    h, st = ops.causal_conv(X, W, Bi)
    q, k, v = (h[..., :nq].reshape(B, T, Hk, Dk), h[..., nq:2 * nq].reshape(B, T, Hk, Dk),
               h[..., 2 * nq:].reshape(B, T, Hv, Dv))
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    y, S = ops.gated_delta_rule(q, k, v, G_, BE, chunk=16)
    o = ops.group_norm(y.reshape(B, T, nv), NW, None, Z, groups=Hv)
    out, S2 = ops.selective_scan(o, rows(SC["dt"]), SC["A"], rows(SC["Bm"]), rows(SC["Cm"]), SC["D"],
                                 rows(SC["z"]), SC["dt_bias"])
    out.backward(dev_of(dy, "f32", cuda))

    # the oracles, composed
    seqs = seqs_of(B, T, None)
    flat = lambda a: a.reshape(B * T, -1)
    hr, _ = L.conv_forward(flat(x), w, b, None, True, seqs)
    qr, kr, vr = (hr[:, i:j].reshape(B, T, H, D) for i, j, H, D in
                  ((0, nq, Hk, Dk), (nq, 2 * nq, Hk, Dk), (2 * nq, C, Hv, Dv)))
    yr, _ = O.forward(qr, kr, vr, g, beta, None)
    orr = L.norm_forward(flat(yr), nw, None, flat(z), Hv, 1e-6, False, True)
    sargs = [s[k] for k in ("dt", "A", "Bm", "Cm", "D", "z", "dt_bias")]
    outr, _ = L.scan_forward(orr, *sargs, None, True, seqs)
    gs = L.scan_backward(orr, *sargs, None, True, seqs, flat(dy))
    dyr, dwr, _, dzr = L.norm_backward(flat(yr), nw, None, flat(z), Hv, 1e-6, False, True, gs["du"])
    dq, dk, dv, dg, db, _ = O.backward(qr, kr, vr, g, beta, dyr.reshape(B, T, Hv, Dv), None, None)
    dh = np.concatenate([flat(dq), flat(dk), flat(dv)], 1)
    dxr, dcw, dcb, _ = L.conv_backward(flat(x), w, b, None, True, seqs, dh)
    # the recurrence's bar for fp32 inputs (relative L2 1e-5), which the
    # stages before and behind it multiply by their condition, at most 10 each
    for name, got, ref in (("out", out, outr), ("dx", X.grad, dxr), ("dw", W.grad, dcw), ("db", Bi.grad, dcb),
                           ("dg", G_.grad, dg), ("dbeta", BE.grad, db), ("dz", Z.grad, dzr),
                           ("dnw", NW.grad, dwr.reshape(Hv, Dv).sum(0)), ("dA", SC["A"].grad, gs["dA"]),
                           ("ddt", SC["dt"].grad, gs["ddt"]), ("dB", SC["Bm"].grad, gs["dB"])):
        err = O.rel_l2(got.detach().double().cpu().numpy().reshape(ref.shape), ref)
        assert err <= 1e-4, (name, err)

    # served: a prompt of 30 tokens, then one by one
    with torch.no_grad():
        window = state = scan = None
        served = []
        for i, j in [(0, 30)] + [(t, t + 1) for t in range(30, T)]:
            h, window = ops.gdr_conv_forward(X[:, i:j].contiguous(), W, Bi, window)
            n = j - i
            q, k, v = (h[..., :nq].reshape(B, n, Hk, Dk), h[..., nq:2 * nq].reshape(B, n, Hk, Dk),
                       h[..., 2 * nq:].reshape(B, n, Hv, Dv))
            y, state, _ = ops.gdr_forward(q.contiguous(), k.contiguous(), v.contiguous(), G_[:, i:j].contiguous(),
                                          BE[:, i:j].contiguous(), state, chunk=16, save=False)
            o, _ = ops.gdr_norm_forward(y.reshape(B, n, nv), NW, None, Z[:, i:j].contiguous(), groups=Hv,
                                        save=False)
            p, scan, _ = ops.gdr_scan_forward(o, rows(SC["dt"], i, j), SC["A"], rows(SC["Bm"], i, j),
                                              rows(SC["Cm"], i, j), SC["D"], rows(SC["z"], i, j), SC["dt_bias"],
                                              scan, save=False)
            served.append(p)
    err = O.rel_l2(torch.cat(served, 1).double().cpu().numpy().reshape(outr.shape), outr)
    assert err <= 1e-4, err
