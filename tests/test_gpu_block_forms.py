"""Forms of linear attention and of the norms around a block that one call
takes alone: a single norm over many rows of a workgroup, and what else the
sizes of the other files do not reach.

Tolerances as in test_gpu_block_ops.py where nothing else is derived.
"""
import numpy as np
import pytest

import oracle.block_oracle as L
from tests.test_gpu_layer_ops import check, dev_of, round_to

pytestmark = pytest.mark.gpu


def ops():
    from gated_delta_rule_recurrence_amd import ops
    return ops


# ---- the norms: one of them, several rows a workgroup ------------------------------

# rows a workgroup of 256, 512 and 1024 lanes takes several of, in either direction
ROWS = ((3000, 600), (1100, 2304), (700, 4104))


def norm_rows(dtype, rows, C, post, pre, center, gate, seed):
    """Rows of very different sizes (2^-6 to 2^6), so that the statistics of
    one show in another's."""
    r = np.random.default_rng(seed)
    size = 2.0 ** r.integers(-6, 7, size=(rows, 1))
    n = lambda: round_to(r.normal(size=(rows, C)) * size, dtype)
    d = dict(x=n(), res=n(), dy=round_to(r.normal(size=(rows, C)), dtype), dh=round_to(r.normal(size=(rows, C)), dtype))
    d["gate"] = round_to(r.normal(size=(rows if gate == "row" else 1, C)), dtype) if gate else None
    w = [round_to(1 + 0.2 * r.normal(size=C), dtype) if use else None for use in (post, pre)]
    b = [round_to(r.normal(size=C), dtype) if center and use else None for use in (post, pre)]
    d["w"] = (w[0], b[0], w[1], b[1])
    return d


@pytest.mark.parametrize("dtype,gate", (("bf16", "row"), ("f32", "channel")))
@pytest.mark.parametrize("post,pre,center", ((0, 1, 0), (1, 0, 0), (0, 1, 1), (1, 0, 1)))
@pytest.mark.parametrize("rows,C", ROWS + ((3100, 1001),))
def test_res_one_norm_many_rows(cuda, rows, C, post, pre, center, dtype, gate):
    import torch
    d = norm_rows(dtype, rows, C, post, pre, center, gate, seed=C + post)
    on = lambda a: dev_of(a, dtype, cuda)
    g = None if d["gate"] is None else on(d["gate"]) if gate == "row" else on(d["gate"])[0]
    args = [on(d["x"]), on(d["res"]), g, *map(on, d["w"])]
    how = dict(alpha=0.6, eps=1e-5, post=bool(post), pre=bool(pre), center=bool(center))
    y, h, stats = ops().gdr_res_forward(*args, **how)
    back = lambda: ops().gdr_res_backward(*args, stats, on(d["dy"]) if pre else None, on(d["dh"]), **how)
    grads = back()
    for _ in range(3):
        again = ops().gdr_res_forward(*args, **how)
        for a, b in zip((y, h, stats, *grads), (*again, *back())):
            assert a is None and b is None or torch.equal(a, b)
    host = (d["x"], d["res"], d["gate"], *d["w"], 0.6, 1e-5, post, pre, center)
    ref, mag = (L.res_forward(*host, mag=m) for m in (False, True))
    if pre:
        check("y", y, ref[0], mag[0], dtype, 128)
    check("h", h, ref[1], mag[1], dtype, 128)
    ref, mag = (L.res_backward(*host, dy=d["dy"], dh=d["dh"], mag=m) for m in (False, True))
    given = (1, 1, g, *d["w"])
    for i, name in enumerate(("dx", "dr", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")):
        if given[i] is None:
            assert grads[i] is None
        else:
            check(name, grads[i], ref[i], mag[i], dtype, 256 + (rows if i >= 2 else 0))


@pytest.mark.parametrize("post,pre,center", ((1, 1, 0), (0, 1, 0), (1, 0, 1)))
@pytest.mark.parametrize("rows,C", ROWS)
def test_res_in_place_many_rows(cuda, rows, C, post, pre, center):
    """h over the residual and y over x, with the next row in flight."""
    import torch
    x, r = (torch.randn(rows, C, device=cuda).bfloat16() for _ in range(2))
    w = torch.rand(C, device=cuda).bfloat16()
    args = (None, w if post else None, None, w if pre else None)
    how = dict(post=bool(post), pre=bool(pre), center=bool(center), save=False)
    y, h, _ = ops().gdr_res_forward(x, r, *args, **how)
    a, b, _ = ops().gdr_res_forward(x, r, *args, **how, y=x if pre else None, h=r)
    assert b is r and torch.equal(r, h) and (not pre or a is x and torch.equal(x, y))


# ---- linear attention: the precision of what is fp32 inside -------------------------

# output: the tensor whose two neighbouring rows cancel, the one that is equal there
PAIRS = {"y": ("v", "k"), "dq": ("k", "v"), "dk": ("q", "dy"), "dv": ("dy", "q")}


def lin_run(on, S0=None, dS_T=None, *, T, scale=1.0, want_dlog_g=True):
    args = [on[n] for n in ("q", "k", "v", "log_g")]
    y, S_T, saved = ops().gdr_lin_forward(*args, S0, scale=scale, T=T)
    grads = ops().gdr_lin_backward(*args, saved, on["dy"], dS_T, want_dlog_g=want_dlog_g)
    return dict(zip(("y", "S_T", "dq", "dk", "dv", "dlog_g", "dS0"), (y, S_T, *grads)))


def lin_ref(d, seqs, S0=None, dS_T=None, scale=1.0):
    host = [d[n] for n in ("q", "k", "v", "log_g")] + [S0, scale, seqs]
    out = []
    for m in (False, True):
        out.append(dict(zip(("y", "S_T"), L.lin_forward(*host, mag=m))))
        out[-1].update(zip(("dq", "dk", "dv", "dlog_g", "dS0"), L.lin_backward(*host, d["dy"], dS_T, mag=m)))
    return out


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("out", PAIRS)
@pytest.mark.parametrize("B,T,H,reps,flow", ((6, 130, 2, 1, True), (6, 130, 1, 2, False), (1, 1100, 1, 1, False)))
def test_lin_terms_that_cancel(cuda, out, dtype, B, T, H, reps, flow):
    """Two steps whose contributions are opposite but for the decay between
    them, 2^-14: what is left of them behind shows every bit that P, uf V or the
    state lose as an operand.  All other factors are positive, so the two steps'
    products are the same bits.  Roundings, each of at most one unit of the
    terms: an exponential (its argument is far below one) 2 and its product 1
    on either side of the decay, at most 5 in the sum of the two terms' three
    pieces, and of fp32 rows the three products that are left out, 3; behind the
    cancellation they are of what is left.  n = 14 (16 with the flows' own term).
    An operand of two pieces is off by up to 64."""
    r = np.random.default_rng(T + reps + len(out))
    Hv, D, rows = H * reps, 64, B * T
    pos = lambda *s: round_to(r.uniform(0.5, 1.0, size=s), dtype)
    d = dict(q=pos(rows, H, D), k=pos(rows, H, D), v=pos(rows, Hv, D), dy=pos(rows, Hv, D))
    lg = -r.uniform(0, 2.0 ** -16, size=(rows, Hv))
    cancel, equal = PAIRS[out]
    only = np.zeros(rows, bool)
    for b in range(B):
        at = b * T + (int(r.integers(1, 60)) if out in ("y", "dq") else T - int(r.integers(3, 60)))
        d[cancel][at + 1] = -d[cancel][at]
        d[equal][at + 1] = d[equal][at]
        lg[at + 1] = -2.0 ** -14 * r.uniform(1, 2, size=Hv)
        only[at:at + 2] = True
    d[cancel][~only] = 0.0
    d["log_g"] = round_to(lg, "f32")
    on = {n: dev_of(a, "f32" if n == "log_g" else dtype, cuda) for n, a in d.items()}
    got = lin_run(on, T=T, want_dlog_g=flow)[out]
    ref, mag = lin_ref(d, [(b * T, (b + 1) * T) for b in range(B)])
    # (the step of the pair that the other has not joined: no cancellation)
    check(out, got, ref[out], mag[out], dtype, 16 if flow else 14)


@pytest.mark.parametrize("out", ("y", "dq", "dk", "dv"))
def test_lin_states_that_cancel(cuda, out):
    """bf16 rows against a given fp32 state whose two contracted entries cancel
    but for 2^-14 of them: at most 5 roundings in their sum, one a tile in the
    state, so n = 8; an operand of two pieces is off by up to 64."""
    r = np.random.default_rng(3)
    B, T, H, D = 3, 100, 2, 64
    zero = np.zeros((B * T, H, D))
    d = dict(q=zero, k=zero, v=zero, dy=zero, log_g=round_to(-r.uniform(0, 0.01, size=(B * T, H)), "f32"))
    # y = S q, dq = S^T dy, dk = D^T v, dv = D k: the rows that the state meets
    row, over_keys, back = {"y": ("q", 1, 0), "dq": ("dy", 0, 0), "dk": ("v", 0, 1), "dv": ("k", 1, 1)}[out]
    x = round_to(r.normal(size=(B * T, H)), "bf16")
    d[row] = zero.copy()
    d[row][..., 5], d[row][..., 40] = x, -x
    S = r.normal(size=(B, H, D, D))
    if over_keys:
        S[..., 40] = S[..., 5] * (1 + 2.0 ** -14 * r.uniform(0.5, 1, size=S[..., 5].shape))
    else:
        S[..., 40, :] = S[..., 5, :] * (1 + 2.0 ** -14 * r.uniform(0.5, 1, size=S[..., 5, :].shape))
    S = round_to(S, "f32")
    S0, dS_T = (None, S) if back else (S, None)
    on = {n: dev_of(a, "f32" if n == "log_g" else "bf16", cuda) for n, a in d.items()}
    for flow in (True, False):
        got = lin_run(on, dev_of(S0, "f32", cuda), dev_of(dS_T, "f32", cuda), T=T, want_dlog_g=flow)[out]
        ref, mag = lin_ref(d, [(b * T, (b + 1) * T) for b in range(B)], S0, dS_T)
        check(out, got, ref[out], mag[out], "bf16", 8)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,Hk,Hv", ((2, 200, 2, 4), (1, 1100, 1, 1), (1, 2000, 1, 2)))
def test_lin_fp32_outputs_as_a_whole(cuda, dtype, B, T, Hk, Hv):
    """The outputs that stay in fp32, by their relative distance from 64 bits.
    A term of a state carries about 2 units (an exponential, a product), and the
    sums of up to 32 tiles six roundings each, of 0.3 units in the mean square:
    4 units; 6e-7 is 10.  The decay's gradient adds up the flows of all later
    steps, of which as many as a decay reaches, 5, make it: T = 200 takes
    sqrt(200 / 5) of the flows' 4 units, 25, T = 2000 80: 6e-6.  Operands of two
    pieces leave more than 1e-6 in the states."""
    r = np.random.default_rng(T)
    D, rows = 64, B * T
    n = lambda *s: round_to(r.normal(size=s), dtype)
    d = dict(q=n(rows, Hk, D), k=n(rows, Hk, D), v=n(rows, Hv, D), dy=n(rows, Hv, D),
             log_g=round_to(-r.exponential(0.2, size=(rows, Hv)), "f32"))
    st = lambda: round_to(r.normal(size=(B, Hv, D, D)), "f32")
    S0, dS_T = st(), st()
    on = {m: dev_of(a, "f32" if m == "log_g" else dtype, cuda) for m, a in d.items()}
    got = lin_run(on, dev_of(S0, "f32", cuda), dev_of(dS_T, "f32", cuda), T=T)
    ref, _ = lin_ref(d, [(b * T, (b + 1) * T) for b in range(B)], S0, dS_T)
    for name, most in (("S_T", 6e-7), ("dS0", 6e-7), ("dlog_g", 6e-6)) + ((("y", 6e-7),) if dtype == "f32" else ()):
        a = got[name].double().cpu().numpy().reshape(ref[name].shape)
        off = float(np.linalg.norm(a - ref[name]) / np.linalg.norm(ref[name]))
        print(name, f"{off:.2e}")
        assert off <= most, name


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T", (60, 200, 700))
def test_lin_outputs_do_not_depend_on_each_other(cuda, dtype, T):
    """y is the same bits whichever other outputs a call is asked for, and so
    are the gradients."""
    import torch
    g = torch.Generator(device=cuda).manual_seed(T)
    n = lambda *s: torch.randn(*s, device=cuda, generator=g)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, dy = (n(1, T, 2, 64).to(t) for _ in range(4))
    lg = -torch.rand(1, T, 2, device=cuda, generator=g)
    y, S, saved = ops().gdr_lin_forward(q, k, v, lg)
    for kw in (dict(save=False), dict(out_state=False), dict(save=False, out_state=False)):
        assert torch.equal(y, ops().gdr_lin_forward(q, k, v, lg, **kw)[0]), kw
    grads = ops().gdr_lin_backward(q, k, v, lg, saved, dy)
    some = ops().gdr_lin_backward(q, k, v, lg, saved, dy, want_dS0=False)
    assert all(torch.equal(a, b) for a, b in zip(grads[:4], some))
