"""GPU parity of linear attention and of the norms around a block against
their float64 oracle, element by element.

Tolerance.  An output element is off by at most
    half |ref| + n 2^-24 mag + 1e-30,
half a rounding step of its type (2^-8 bf16, 0 for what stays in fp32, whose
store is among the n), mag the sum of the absolute values of its terms (the
oracle's mag=True), n the roundings in fp32 on the way to it:
  * linear attention: a decay between two steps is one exponential of a sum
    formed in 64 bits (its argument rounds once, by |x| units that e^x weighs
    with at most 0.37: 4 units), or a product of single steps' (4 units each).
    Products of matrices whose fp32 operand is held in two bf16 pieces (bf16
    rows) are off by 2^-18 of each term, 64 units; it happens to the products
    of queries and keys and to the states: 128.  Sums of up to 256 terms and
    the joins of chunks: 8 a step at most.  n = 256 + 8 steps; twice that for
    the decay's gradient, which sums products of two such.
  * norms: sums of 8 terms a lane, then a tree of 10: a statistic is off by 32
    units, either norm by 64; the backward runs through both: n = 128 and 256,
    plus one per row in the sums over rows.
"""
import numpy as np
import pytest

import oracle.block_oracle as L
from tests.test_gpu_layer_ops import PACKED, PACKED_ROWS, check, dev_of, dev_spans, outside, round_to, seqs_of, spoil

pytestmark = pytest.mark.gpu


def ops():
    from gated_delta_rule_recurrence_amd import ops
    return ops


def wide(t, tail, pad=8):
    """The same rows as a slice of wider ones (a row stride), NaN around."""
    import torch
    if t is None:
        return None
    lead = t.shape[:t.dim() - tail]
    flat = t.reshape(*lead, -1)
    w = torch.full((*lead, flat.shape[-1] + 3 * pad), float("nan"), dtype=t.dtype, device=t.device)
    w[..., pad:pad + flat.shape[-1]] = flat
    s = w[..., pad:pad + flat.shape[-1]]
    return s.unflatten(-1, t.shape[t.dim() - tail:])


# ---- linear attention -----------------------------------------------------------

def lin_data(dtype, rows, B, Hk, Hv, Dk, Dv, decay="step", gdtype="f32", state=True, seed=0, rate=0.2):
    r = np.random.default_rng(seed)
    n = lambda *s: round_to(r.normal(size=s), dtype)
    d = dict(q=n(rows, Hk, Dk), k=round_to(r.normal(size=(rows, Hk, Dk)) * Dk ** -0.5, dtype), v=n(rows, Hv, Dv),
             dy=n(rows, Hv, Dv))
    d["log_g"] = {"step": lambda: round_to(-r.exponential(rate, size=(rows, Hv)), gdtype),
                  "head": lambda: round_to(-r.exponential(rate, size=Hv), gdtype),
                  "none": lambda: None}[decay]()
    st = lambda: round_to(r.normal(size=(B, Hv, Dv, Dk)) * 0.3, "f32")
    d["S0"], d["dS_T"] = (st(), st()) if state else (None, None)
    return d


def lin_case(dev, dtype, B, T, Hk, Hv, Dk, Dv, *, decay="step", gdtype="f32", state=True, spans=None, rows=None,
             stride=False, seed=0, rate=0.2, log_g=None, scale=0.7):
    rows = B * T if rows is None else rows
    d = lin_data(dtype, rows, B, Hk, Hv, Dk, Dv, decay, gdtype, state, seed, rate)
    if log_g is not None:
        d["log_g"] = log_g
    seqs = seqs_of(B, T, spans)
    longest = T if spans is None else max([j - i for i, j in seqs] + [0])
    on = {n: dev_of(d[n], dtype, dev) for n in ("q", "k", "v", "dy")}
    on["log_g"] = dev_of(d["log_g"], gdtype, dev)
    for n in ("q", "k", "v", "dy") + (("log_g",) if decay == "step" else ()):
        spoil(on[n], seqs)
    if stride:
        for n in ("q", "k", "v"):
            on[n] = wide(on[n], 2)
        if decay == "step":
            on["log_g"] = wide(on["log_g"], 1)
    args = [on[n] for n in ("q", "k", "v", "log_g")]
    S0, dS_T = dev_of(d["S0"], "f32", dev), dev_of(d["dS_T"], "f32", dev)
    kw = dict(scale=scale, spans=dev_spans(spans, dev), T=longest)
    y, S_T, saved = ops().gdr_lin_forward(*args, S0, **kw)
    grads = ops().gdr_lin_backward(*args, saved, on["dy"], dS_T)
    y2, S2, none = ops().gdr_lin_forward(*args, S0, save=False, **kw)
    assert none is None and bool((y2 == y).all()) and bool((S2 == S_T).all())
    n = 256 + 8 * longest
    host = [d[x] for x in ("q", "k", "v", "log_g", "S0")] + [scale, seqs]
    ref, mag = (L.lin_forward(*host, mag=m) for m in (False, True))
    check("y", y, ref[0], mag[0], dtype, n)
    check("S_T", S_T, ref[1], mag[1], "f32", n)
    ref, mag = (L.lin_backward(*host, d["dy"], d["dS_T"], mag=m) for m in (False, True))
    reps = Hv // Hk
    for name, i, ty in (("dq", 0, dtype), ("dk", 1, dtype), ("dv", 2, dtype), ("dlog_g", 3, gdtype), ("dS0", 4, "f32")):
        if ref[i] is None:
            assert grads[i] is None
            continue
        more = (2 * n + (rows if decay == "head" else 0)) if name == "dlog_g" else n + reps
        check(name, grads[i], ref[i], mag[i], ty, more)
    out = outside(rows, seqs)
    for t in (y, *grads[:3]) + ((grads[3],) if decay == "step" else ()):
        assert not t.reshape(rows, -1)[out].any()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("T", (1, 2, 15, 16, 17, 63, 64, 65, 127, 200))
def test_lin_lengths(cuda, dtype, T):
    lin_case(cuda, dtype, 2, T, 2, 4, 64, 64, seed=T)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", ((1, 1, 1, 1), (2, 6, 37, 53), (1, 3, 128, 128), (3, 3, 192, 128), (1, 2, 256, 256),
                                         (1, 8, 128, 64), (2, 2, 8, 200), (2, 4, 100, 24), (1, 5, 16, 16), (1, 2, 96, 160)))
def test_lin_widths(cuda, dtype, Hk, Hv, Dk, Dv):
    lin_case(cuda, dtype, 2, 70, Hk, Hv, Dk, Dv, seed=Dk + Dv)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("Dk,Dv", ((64, 64), (33, 40), (128, 128)))
def test_lin_packed(cuda, dtype, Dk, Dv):
    lin_case(cuda, dtype, len(PACKED), 0, 2, 4, Dk, Dv, spans=PACKED, rows=PACKED_ROWS)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_lin_one_long_sequence(cuda, dtype):
    """Long enough that the sequence is cut and joined."""
    lin_case(cuda, dtype, 1, 1100, 1, 2, 64, 32, rate=0.01)


def test_lin_long_packed(cuda):
    lin_case(cuda, "bf16", 4, 0, 1, 2, 64, 64, spans=[(3, 700), (700, 701), (701, 701), (710, 1500)], rows=1510, rate=0.02)


@pytest.mark.parametrize("kw", (dict(decay="head"), dict(decay="none"), dict(gdtype="bf16"), dict(state=False),
                                dict(stride=True), dict(scale=1.0), dict(scale=-2.5), dict(decay="head", gdtype="bf16"),
                                dict(rate=5.0), dict(rate=0.0)))
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_lin_options(cuda, dtype, kw):
    lin_case(cuda, dtype, 2, 90, 2, 4, 64, 48, seed=3, **kw)


def test_lin_odd_stride(cuda):
    """Rows that begin on no vector's boundary but the first."""
    import torch
    r = np.random.default_rng(5)
    T, H, D = 40, 2, 17
    buf = torch.from_numpy(r.normal(size=(T, 3 * H * D + 1)).astype(np.float32)).to(cuda)
    q = buf[:, :H * D].unflatten(-1, (H, D))
    k, v = (buf[:, :H * D].clone().unflatten(-1, (H, D)) * s for s in (0.5, 0.25))
    y, S, _ = ops().gdr_lin_forward(q, k, v, None, T=T)
    host = [x.double().cpu().numpy() for x in (q, k, v)]
    ref, mag = (L.lin_forward(*host, None, None, 1.0, [(0, T)], mag=m) for m in (False, True))
    check("y", y, ref[0], mag[0], "f32", 256 + 8 * T)
    check("S_T", S, ref[1], mag[1], "f32", 256 + 8 * T)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_lin_decays_that_forget(cuda, dtype):
    """log_g of -inf at some steps, very negative and positive ones at others:
    the state before a forgetting step reaches nothing behind it."""
    r = np.random.default_rng(6)
    lg = -r.exponential(0.1, size=(2 * 150, 4))
    lg[r.random(lg.shape) < 0.05] = -np.inf
    lg[r.random(lg.shape) < 0.02] = -300.0
    lg[r.random(lg.shape) < 0.05] = 0.3
    lin_case(cuda, dtype, 2, 150, 2, 4, 64, 64, log_g=round_to(lg, "f32"), seed=7)


def test_lin_small_decay_gradients(cuda):
    """Strong decays: what crosses a step is e^-12 of what stays, and its
    gradient is still right relative to itself."""
    import torch
    d = lin_data("f32", 130, 1, 1, 2, 32, 32, state=False, seed=8)
    d["log_g"] = np.full((130, 2), -12.0)
    on = [dev_of(d[n], "f32", cuda) for n in ("q", "k", "v", "log_g")]
    _, _, saved = ops().gdr_lin_forward(*on, T=130)
    dg = ops().gdr_lin_backward(*on, saved, dev_of(d["dy"], "f32", cuda))[3]
    ref = L.lin_backward(d["q"], d["k"], d["v"], d["log_g"], None, 1.0, [(0, 130)], d["dy"], None)[3]
    assert float(np.linalg.norm(dg.double().cpu().numpy() - ref) / np.linalg.norm(ref)) < 1e-4
    assert torch.isfinite(dg).all()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_lin_tokens_follow_the_prompt(cuda, dtype):
    """A prompt, then single tokens with the state in place, against one pass."""
    import torch
    B, T, n = 3, 70, 5
    d = lin_data(dtype, B * (T + n), B, 2, 4, 64, 48, seed=9)
    on = {m: dev_of(d[m], dtype, cuda).view(B, T + n, *d[m].shape[1:]) for m in ("q", "k", "v")}
    lg = dev_of(d["log_g"], "f32", cuda).view(B, T + n, -1)
    S0 = dev_of(d["S0"], "f32", cuda)
    y, S, _ = ops().gdr_lin_forward(on["q"], on["k"], on["v"], lg, S0, scale=0.5, save=False)
    cut = lambda i, j: [x[:, i:j].contiguous() for x in (on["q"], on["k"], on["v"], lg)]
    ys, st, _ = ops().gdr_lin_forward(*cut(0, T), S0, scale=0.5, save=False)
    out = [ys]
    for t in range(T, T + n):
        yt, same, _ = ops().gdr_lin_forward(*cut(t, t + 1), st, scale=0.5, save=False, S_T=st)
        assert same is st
        out.append(yt)
    host = [d[m] for m in ("q", "k", "v", "log_g", "S0")] + [0.5, seqs_of(B, T + n, None)]
    ref, mag = (L.lin_forward(*host, mag=m) for m in (False, True))
    for name, a, b in (("y", y, torch.cat(out, 1)), ("S_T", S, st)):
        i = 0 if name == "y" else 1
        for got in (a, b):
            check(name, got, ref[i], mag[i], dtype if i == 0 else "f32", 256 + 8 * (T + n))


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("T", (1, 3, 8, 9))
def test_lin_few_steps(cuda, dtype, T):
    for Dk, Dv in ((128, 128), (64, 256), (36, 20), (7, 130)):
        lin_case(cuda, dtype, 5, T, 2, 4, Dk, Dv, seed=T)


@pytest.mark.parametrize("seed", range(12))
def test_lin_random_shapes(cuda, seed):
    r = np.random.default_rng(100 + seed)
    Hk = int(r.integers(1, 4))
    dims = [int(r.choice((8, 16, 64, 128, int(r.integers(1, 257))))) for _ in range(2)]
    dtype = str(r.choice(("f32", "bf16")))
    kw = dict(decay=str(r.choice(("step", "head", "none"))), gdtype=str(r.choice(("f32", "bf16"))),
              state=bool(r.random() < 0.5), stride=bool(r.random() < 0.4), rate=float(r.choice((0.01, 0.2, 2.0))), seed=seed)
    if r.random() < 0.5:
        rows = int(r.integers(20, 260))
        at = np.sort(r.integers(0, rows + 1, size=6))
        lin_case(cuda, dtype, 3, 0, Hk, Hk * int(r.integers(1, 4)), *dims, rows=rows,
                 spans=[(int(at[2 * i]), int(at[2 * i + 1])) for i in range(3)], **kw)
    else:
        lin_case(cuda, dtype, int(r.integers(1, 4)), int(r.integers(1, 200)), Hk, Hk * int(r.integers(1, 4)), *dims, **kw)


# ---- the norms around a block -----------------------------------------------------

def res_case(dev, dtype, B, T, C, *, rdtype=None, wdtype=None, gdtype=None, gate="none", post=True, pre=True,
             center=False, offset=0.0, weights=True, stride=False, dh=True, alpha=0.6, seed=0):
    import torch
    rdtype, wdtype, gdtype = rdtype or dtype, wdtype or dtype, gdtype or dtype
    r = np.random.default_rng(seed)
    rows = B * T
    n = lambda ty, *s: round_to(r.normal(size=s), ty)
    x, res, dy, dhv = n(dtype, rows, C), n(rdtype, rows, C), n(dtype, rows, C), n(rdtype, rows, C)
    k = {"none": 0, "channel": 1, "sequence": B, "row": rows}[gate]
    g = n(gdtype, k, C) if k else None
    w = [round_to(1 + 0.2 * r.normal(size=C) - offset, wdtype) if weights and use else None for use in (post, pre)]
    b = [n(wdtype, C) if weights and center and use else None for use in (post, pre)]
    shape = {"none": None, "channel": (C,), "sequence": (B, C), "row": (B, T, C)}[gate]
    xd, rd = (dev_of(a, t, dev).view(B, T, C) for a, t in ((x, dtype), (res, rdtype)))
    gd = None if g is None else dev_of(g, gdtype, dev).view(shape)
    if stride:
        xd, rd = wide(xd, 1), wide(rd, 1)
        gd = wide(gd, 1) if gate in ("sequence", "row") else gd
    args = [xd, rd, gd, *[dev_of(a, wdtype, dev) for a in (w[0], b[0], w[1], b[1])]]
    how = dict(alpha=alpha, eps=1e-5, post=post, pre=pre, center=center, weight_offset=offset)
    y, h, stats = ops().gdr_res_forward(*args, **how)
    grads = ops().gdr_res_backward(*args, stats, dev_of(dy, dtype, dev).view(B, T, C) if pre else None,
                                   dev_of(dhv, rdtype, dev).view(B, T, C) if dh else None, **how)
    y2, h2, none = ops().gdr_res_forward(*args, save=False, **how)
    assert none is None and torch.equal(h, h2) and (y is None or torch.equal(y, y2))
    host = (x, res, g, w[0], b[0], w[1], b[1], alpha, 1e-5, post, pre, center)
    ref, mag = (L.res_forward(*host, offset=offset, mag=m) for m in (False, True))
    if pre:
        check("y", y, ref[0], mag[0], dtype, 128)
    else:
        assert y is None
    check("h", h, ref[1], mag[1], rdtype, 128)
    ref, mag = (L.res_backward(*host, dy=dy, dh=dhv if dh else None, offset=offset, mag=m) for m in (False, True))
    given = (x, res, g, w[0], b[0], w[1], b[1])
    for i, (name, ty) in enumerate((("dx", dtype), ("dr", rdtype), ("dgate", gdtype), ("dpost_w", wdtype),
                                    ("dpost_b", wdtype), ("dpre_w", wdtype), ("dpre_b", wdtype))):
        if given[i] is None:
            assert grads[i] is None
            continue
        check(name, grads[i], ref[i], mag[i], ty, 256 + (rows if i >= 2 else 0))


@pytest.mark.parametrize("dtype,rdtype", (("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")))
@pytest.mark.parametrize("C", (1, 8, 31, 64, 200, 512, 520, 1110, 2048, 2056, 4096, 5120, 8192))
def test_res_widths(cuda, dtype, rdtype, C):
    res_case(cuda, dtype, 2, 5, C, rdtype=rdtype, gate="channel", seed=C)


@pytest.mark.parametrize("gate", ("none", "channel", "sequence", "row"))
@pytest.mark.parametrize("post,pre,center", ((1, 1, 0), (0, 1, 0), (1, 0, 0), (1, 1, 1), (0, 1, 1), (1, 0, 1), (0, 0, 0)))
@pytest.mark.parametrize("C", (72, 1000))
def test_res_options(cuda, gate, post, pre, center, C):
    for dtype in ("f32", "bf16"):
        res_case(cuda, dtype, 3, 11, C, gate=gate, post=bool(post), pre=bool(pre), center=bool(center), seed=C)


@pytest.mark.parametrize("kw", (dict(wdtype="f32"), dict(gdtype="f32"), dict(gdtype="f32", gate="row"), dict(offset=1.0),
                                dict(weights=False), dict(stride=True), dict(stride=True, gate="row"), dict(dh=False),
                                dict(rdtype="f32", stride=True), dict(wdtype="f32", rdtype="f32", offset=1.0, center=True),
                                dict(alpha=0.0), dict(alpha=-1.5, center=True, weights=False)))
def test_res_mixed(cuda, kw):
    res_case(cuda, "bf16", 2, 9, 328, **{"gate": "sequence", **kw})
    res_case(cuda, "bf16", 2, 9, 1304, **{"gate": "sequence", **kw})


@pytest.mark.parametrize("B,T,C", ((1, 1, 64), (1, 5000, 64), (700, 3, 64), (3, 2000, 96), (1, 1300, 1024), (40, 30, 1024),
                                   (2000, 2, 600), (5, 701, 520)))
@pytest.mark.parametrize("gate", ("channel", "sequence", "row"))
def test_res_rows(cuda, B, T, C, gate):
    """Gate rows of one workgroup, of several, and several in one."""
    res_case(cuda, "bf16", B, T, C, gate=gate, wdtype="f32", gdtype="f32", seed=B)


def test_res_odd_stride(cuda):
    """Rows that begin on no vector's boundary but the first."""
    import torch
    r = np.random.default_rng(2)
    buf = torch.from_numpy(r.normal(size=(37, 129)).astype(np.float32)).to(cuda)
    x = buf[:, :64]
    y, h, _ = ops().gdr_res_forward(x, x)
    xd = x.double().cpu().numpy()
    host = (xd, xd, None, None, None, None, None, 1.0, 1e-6, 1, 1, 0)
    ref, mag = (L.res_forward(*host, mag=m) for m in (False, True))
    check("y", y, ref[0], mag[0], "f32", 128)
    check("h", h, ref[1], mag[1], "f32", 128)


def test_res_in_place(cuda):
    """h over the residual and y over x."""
    import torch
    for C in (64, 1000, 4096):
        x, r = (torch.randn(50, C, device=cuda).bfloat16() for _ in range(2))
        w = torch.rand(C, device=cuda).bfloat16()
        y, h, _ = ops().gdr_res_forward(x, r, None, w, None, w, save=False)
        a, b, _ = ops().gdr_res_forward(x, r, None, w, None, w, save=False, y=x, h=r)
        assert a is x and b is r and torch.equal(x, y) and torch.equal(r, h)


@pytest.mark.parametrize("center", (False, True))
def test_res_rows_of_zeros(cuda, center):
    """A row that the block and the residual leave empty: eps alone under the root."""
    import torch
    x, r = torch.zeros(4, 256, device=cuda), torch.zeros(4, 256, device=cuda)
    w = torch.ones(256, device=cuda)
    y, h, stats = ops().gdr_res_forward(x, r, None, w, None, w, center=center)
    assert not y.any() and not h.any() and torch.isfinite(stats).all()
    grads = ops().gdr_res_backward(x, r, None, w, None, w, None, stats, torch.ones_like(x), torch.ones_like(x), center=center)
    assert all(torch.isfinite(g).all() for g in grads if g is not None)
