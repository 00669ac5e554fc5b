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


# ---- linear attention: decays that grow, decays that forget --------------------------

def lin_zero(d, names, rows):
    for n in names:
        d[n][rows] = 0.0


def lin_grow_case(cuda, dtype, B, T, H, D, make, S0=None, dS_T=None, outs=("y", "S_T"), skip=0, rate=0.05, seed=0):
    """One call on inputs that make(r, d, first row of a sequence) edits, against
    64 bits wherever the result and its terms are far inside fp32's range.  The
    first `skip` rows of dk and dv are left out: there the adjoint itself passes it."""
    import torch
    r = np.random.default_rng(seed)
    rows = B * T
    n = lambda *s: round_to(r.normal(size=s), dtype)
    d = dict(q=n(rows, H, D), k=round_to(r.normal(size=(rows, H, D)) * D ** -0.5, dtype), v=n(rows, H, D), dy=n(rows, H, D),
             log_g=-r.exponential(rate, size=(rows, H)))
    for b in range(B):
        make(r, d, b * T)
    d["log_g"] = round_to(d["log_g"], "f32")
    S0, dS_T = (None if f is None else round_to(f(r, (B, H, D, D)), "f32") for f in (S0, dS_T))
    on = {m: dev_of(a, "f32" if m == "log_g" else dtype, cuda) for m, a in d.items()}
    got = lin_run(on, dev_of(S0, "f32", cuda), dev_of(dS_T, "f32", cuda), T=T)
    with np.errstate(over="ignore", invalid="ignore"):
        ref, mag = lin_ref(d, [(b * T, (b + 1) * T) for b in range(B)], S0, dS_T)
    for name in outs:
        a, m = ref[name], mag[name]
        g = got[name].double().cpu().numpy().reshape(a.shape)
        inside = m < 1e30
        if name in ("dk", "dv"):
            inside &= (np.arange(rows) % T >= skip)[:, None, None]
        assert inside.mean() > 0.2, name
        ty = "f32" if name in ("S_T", "dS0", "dlog_g") else dtype
        check(name, torch.from_numpy(g[inside]), a[inside], m[inside], ty, (256 + 8 * T) * (2 if name == "dlog_g" else 1))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,H,D", ((2, 130, 2, 64), (1, 1100, 1, 48), (1, 200, 1, 192)))
@pytest.mark.parametrize("steps,each", ((40, 3.0), (1, 100.0), (2, 700.0), (20, 30.0), (64, 2.0), (5, 80.0)))
def test_lin_growth_of_an_empty_state(cuda, dtype, B, T, H, D, steps, each):
    """Decays that grow past fp32's range before there is a state: it stays 0,
    and what comes behind is as without them."""
    def make(r, d, at):
        d["log_g"][at:at + steps] = each
        lin_zero(d, ("k", "v"), slice(at, at + steps - 1))  # (the last step writes)
    lin_grow_case(cuda, dtype, B, T, H, D, make, outs=("y", "S_T", "dq", "dv", "dk"), skip=steps, seed=steps)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,H,D", ((2, 130, 2, 64), (1, 1100, 1, 48)))
def test_lin_growth_of_an_empty_adjoint(cuda, dtype, B, T, H, D):
    """The same at the sequence's end, where no gradient comes from."""
    def make(r, d, at):
        d["log_g"][at + T - 40:at + T] = 3.0
        lin_zero(d, ("q", "dy"), slice(at + T - 40, at + T))
    lin_grow_case(cuda, dtype, B, T, H, D, make, outs=("dk", "dv", "dS0"), S0=lambda r, s: r.normal(size=s), seed=1)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,H,D,steps", ((2, 130, 2, 64, 50), (1, 1100, 1, 48, 50), (1, 1100, 1, 48, 400), (1, 300, 1, 160, 50)))
def test_lin_growth_of_a_small_state(cuda, dtype, B, T, H, D, steps):
    """1e-24 grows by e^100, in one tile or over several segments."""
    def make(r, d, at):
        lin_zero(d, ("v",), slice(at, at + T))
        d["log_g"][at + 3:at + 3 + steps] = 100.0 / steps
    lin_grow_case(cuda, dtype, B, T, H, D, make, S0=lambda r, s: 1e-24 * r.normal(size=s), outs=("y", "S_T", "dq"), rate=0.0, seed=2)

    def back(r, d, at):
        lin_zero(d, ("dy",), slice(at, at + T))
        d["log_g"][at + 3:at + 3 + steps] = 100.0 / steps
    lin_grow_case(cuda, dtype, B, T, H, D, back, dS_T=lambda r, s: 1e-24 * r.normal(size=s), outs=("dk", "dv", "dS0"), rate=0.0, seed=3)

    def steps_of(r, d, at):  # small steps, no state
        d["v"][at:at + 3] *= 2.0 ** -80
        d["v"][at + 3:at + T] = 0.0
        d["log_g"][at + 3:at + 3 + steps] = 100.0 / steps
    lin_grow_case(cuda, dtype, B, T, H, D, steps_of, outs=("y", "S_T", "dq"), rate=0.0, seed=4)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,H,D", ((2, 130, 2, 64), (1, 1100, 1, 48), (3, 8, 2, 64)))
@pytest.mark.parametrize("each,steps", ((4.0, 60), (0.9, 600)))
def test_lin_forgotten_states_stay_forgotten(cuda, dtype, B, T, H, D, each, steps):
    """A log_g of -inf, then growth by more than e^200 with nothing new: what
    was forgotten does not come back, in the tile or over segments."""
    def make(r, d, at):
        on = slice(at + 4, min(at + 4 + steps, at + T))
        d["log_g"][at + 3] = -np.inf
        d["log_g"][on] = each
        lin_zero(d, ("v",), slice(at + 3, on.stop))
    lin_grow_case(cuda, dtype, B, T, H, D, make, S0=lambda r, s: r.normal(size=s), outs=("y", "S_T", "dq"), seed=5)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_lin_strong_decay_and_growth_meet(cuda, dtype):
    """A decay of e^-80 and then growth by e^120 leave e^40."""
    def make(r, d, at):
        lin_zero(d, ("v",), slice(at, at + 130))
        d["log_g"][at + 3] = -80.0
        d["log_g"][at + 4:at + 54] = 2.4
    lin_grow_case(cuda, dtype, 2, 130, 2, 64, make, S0=lambda r, s: r.normal(size=s), outs=("y", "S_T", "dq"), rate=0.0, seed=6)


@pytest.mark.parametrize("T", (1, 5, 8))
def test_lin_growth_of_single_tokens(cuda, T):
    """One step of e^100 (past fp32's range) on a state of 0 and on one of 1e-30."""
    def make(r, d, at):
        d["log_g"][at] = 100.0
    lin_grow_case(cuda, "f32", 3, T, 2, 64, make, outs=("y", "S_T"), seed=7)
    lin_grow_case(cuda, "f32", 3, T, 2, 64, make, S0=lambda r, s: 1e-30 * r.normal(size=s), outs=("y", "S_T"), seed=8)


@pytest.mark.parametrize("T", (4, 100))
def test_lin_infinite_growth_is_not_finite(cuda, T):
    """A log_g of +inf or NaN: the rows before it as without, those from it on
    not finite."""
    import torch
    g = torch.Generator(device=cuda).manual_seed(1)
    q, k, v = (torch.randn(1, T, 2, 64, device=cuda, generator=g) for _ in range(3))
    lg = -torch.rand(1, T, 2, device=cuda, generator=g)
    y0, _, _ = ops().gdr_lin_forward(q, k, v, lg)
    for bad in (float("inf"), float("nan")):
        for at in (T // 2, T - 1):
            odd = lg.clone()
            odd[0, at, 1] = bad
            y, S, _ = ops().gdr_lin_forward(q, k, v, odd)
            assert torch.equal(y[:, :at], y0[:, :at]) and torch.equal(y[:, :, 0], y0[:, :, 0])
            assert not torch.isfinite(y[0, at:, 1]).any() and not torch.isfinite(S[0, 1]).any() and torch.isfinite(S[0, 0]).all()


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,Hk,Hv,D,head", ((2, 130, 2, 4, 64, False), (1, 1100, 1, 2, 48, False), (2, 70, 1, 2, 128, True),
                                              (1, 90, 1, 1, 192, False)))
def test_lin_growth_in_earnest(cuda, dtype, B, T, Hk, Hv, D, head):
    """States and adjoints that grow by e^55 within fp32's range, every output
    of it: tiles of several passes, their flows and the sums over heads."""
    from tests.test_gpu_block_ops import lin_case
    r = np.random.default_rng(T)
    if head:
        lg = r.uniform(0.7, 0.78, size=Hv)
    else:
        lg = -r.exponential(0.01, size=(B * T, Hv))
        for b in range(B):
            lg[b * T + 4:b * T + 59] = r.uniform(0.9, 1.1, size=(55, Hv))
    lin_case(cuda, dtype, B, T, Hk, Hv, D, D, log_g=round_to(lg, "f32"), decay="head" if head else "step", seed=T)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_lin_values_that_are_not_finite_in_a_growing_tile(cuda, dtype):
    """Values that are not finite in the second pass over a tile: the rows
    before them and the other columns as without."""
    import torch
    g = torch.Generator(device=cuda).manual_seed(2)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = lambda *s: torch.randn(*s, device=cuda, generator=g).to(t)
    q, k, v = n(1, 90, 1, 64), n(1, 90, 1, 64), n(1, 90, 1, 64)
    lg = torch.full((1, 90, 1), -0.1, device=cuda)
    lg[:, 2:40] = 2.0
    y0, S0, _ = ops().gdr_lin_forward(q, k, v, lg)
    assert torch.isfinite(y0).all()
    for at in (0, 25, 39, 70):
        odd = v.clone()
        odd[0, at, 0, 7] = float("inf")
        odd[0, at + 1, 0, 50] = float("nan")
        y, S, _ = ops().gdr_lin_forward(q, k, odd, lg)
        for c, i in ((7, at), (50, at + 1)):
            assert torch.equal(y[0, :i, 0, c], y0[0, :i, 0, c]) and not torch.isfinite(y[0, i:, 0, c]).any()
            assert not torch.isfinite(S[0, 0, c]).any()
        rest = [c for c in range(64) if c not in (7, 50)]
        assert torch.equal(y[..., rest], y0[..., rest]) and torch.equal(S[:, :, rest], S0[:, :, rest])


# ---- linear attention: the decay's gradient at strong steps ---------------------------

@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("B,T,H", ((2, 130, 2), (1, 700, 1)))
def test_lin_decay_gradient_of_strong_steps(cuda, dtype, B, T, H):
    """Single steps of -12, -110, -300 and -inf among weak ones.  Where exp is 0
    in fp32 nothing flows; elsewhere the gradient is off by units of the flows
    behind the step (the oracle's mag): a flow carries 16 units (as where terms
    cancel above) and the 64 products of its sum, the suffix sum is in 64 bits,
    and the result rounds once: n = 84."""
    import torch
    r = np.random.default_rng(T)
    rows, D = B * T, 64
    n = lambda *s: round_to(r.normal(size=s), dtype)
    d = dict(q=n(rows, H, D), k=round_to(r.normal(size=(rows, H, D)) * D ** -0.5, dtype), v=n(rows, H, D), dy=n(rows, H, D),
             log_g=-r.exponential(0.01, size=(rows, H)))
    strong = r.choice(rows, size=rows // 12, replace=False)
    d["log_g"][strong] = r.choice((-12.0, -110.0, -300.0, -np.inf), size=(len(strong), H))
    d["log_g"] = round_to(d["log_g"], "f32")
    st = lambda: round_to(r.normal(size=(B, H, D, D)), "f32")
    S0, dS_T = st(), st()
    on = {m: dev_of(a, "f32" if m == "log_g" else dtype, cuda) for m, a in d.items()}
    dg = lin_run(on, dev_of(S0, "f32", cuda), dev_of(dS_T, "f32", cuda), T=T)["dlog_g"]
    ref, mag = lin_ref(d, [(b * T, (b + 1) * T) for b in range(B)], S0, dS_T)
    check("dlog_g", dg, ref["dlog_g"], mag["dlog_g"], "f32", 84)
    gone = torch.from_numpy(d["log_g"] < -104).to(cuda)
    assert gone.any() and not dg.reshape(rows, H)[gone].any()


# ---- no rows, no sequences --------------------------------------------------------------

@pytest.mark.parametrize("wdtype", ("bf16", "f32"))
@pytest.mark.parametrize("C", (64, 600, 2304, 8192))
def test_res_parameters_of_no_rows(cuda, C, wdtype):
    """The C call writes zeros into the parameters' gradients of no rows."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    t = torch.bfloat16 if wdtype == "bf16" else torch.float32
    shape = _lib.GdrResShape(0, C, 0, 0, 0, 0, 1.0, 1e-6, 0.0, _lib.GDR_BF16, _lib.GDR_BF16,
                             _lib.GDR_BF16 if wdtype == "bf16" else _lib.GDR_F32, _lib.GDR_BF16, 1, 1, 1)
    nbytes = _lib.size_of("gdr_res_backward_workspace_bytes", shape)
    ws = torch.full((max(nbytes, 1),), 255, dtype=torch.uint8, device=cuda)
    w = torch.ones(C, dtype=t, device=cuda)
    grads = [torch.full((C,), float("nan"), dtype=t, device=cuda) for _ in range(4)]
    ptrs = [0, 0, 0] + [w.data_ptr()] * 4 + [0] * 6 + [g.data_ptr() for g in grads] + [ws.data_ptr()]
    assert _lib.layer_raw("gdr_res_backward", shape, ptrs, torch.cuda.current_stream().cuda_stream, nbytes) == 0
    assert not any(g.any() for g in grads)
    x = torch.zeros(0, 5, C, device=cuda, requires_grad=True)
    ps = [torch.ones(C, device=cuda, requires_grad=True) for _ in range(2)]
    y, h = ops().residual_norm(x, x, None, ps[0], None, ps[1])
    (y.sum() + h.sum()).backward()
    assert not any(p.grad.any() for p in ps)


@pytest.mark.parametrize("gdtype", ("bf16", "f32"))
def test_lin_decay_per_head_of_no_sequences(cuda, gdtype):
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    t = torch.bfloat16 if gdtype == "bf16" else torch.float32
    Hv = 300
    shape = _lib.GdrLinShape(0, 0, 0, 1, Hv, 16, 16, 0, 0, 0, 0, 1.0, _lib.GDR_F32,
                             _lib.GDR_BF16 if gdtype == "bf16" else _lib.GDR_F32, 1)
    nbytes = _lib.size_of("gdr_lin_backward_workspace_bytes", shape)
    ws = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=cuda)
    lg = torch.zeros(Hv, dtype=t, device=cuda)
    dg = torch.full((Hv,), float("nan"), dtype=t, device=cuda)
    ptrs = [0, 0, 0, lg.data_ptr(), 0, 0, 0, 0, 0, 0, 0, dg.data_ptr(), 0, ws.data_ptr()]
    assert _lib.layer_raw("gdr_lin_backward", shape, ptrs, torch.cuda.current_stream().cuda_stream, nbytes) == 0
    assert not dg.any()


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T", (7, 100, 700))
@pytest.mark.parametrize("bad", (float("nan"), float("inf")))
def test_lin_decays_that_are_not_finite_backward(cuda, dtype, T, bad):
    """A log_g that is not finite at step t reaches dk and dv of the steps before
    t and dq from t on, in its head, and no others (not t's own dk and dv)."""
    import torch
    g = torch.Generator(device=cuda).manual_seed(T)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, dy = (torch.randn(2, T, 2, 64, device=cuda, generator=g).to(t) for _ in range(4))
    lg = -torch.rand(2, T, 2, device=cuda, generator=g)
    grads = lambda lg: ops().gdr_lin_backward(q, k, v, lg, ops().gdr_lin_forward(q, k, v, lg)[2], dy)
    clean = grads(lg)
    for at in sorted({0, 1, T // 2, T - 1}):
        odd = lg.clone()
        odd[1, at, 0] = bad
        got = grads(odd)
        for i, (a, b) in enumerate(zip(got[:3], clean[:3])):  # dq, dk, dv
            reached = torch.zeros(2, T, 2, dtype=torch.bool, device=cuda)
            reached[1, at:, 0] = i == 0
            reached[1, :at, 0] = i > 0
            assert torch.equal(a[~reached], b[~reached]), (at, i)
            assert not torch.isfinite(a[reached]).any(), (at, i)
        assert torch.equal(got[3][0], clean[3][0]) and torch.equal(got[3][1, :, 1], clean[3][1, :, 1])
        assert torch.equal(got[4][0], clean[4][0]) and torch.equal(got[4][1, 1], clean[4][1, 1])
        assert not torch.isfinite(got[4][1, 0]).any()
