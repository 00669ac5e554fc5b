"""Linear attention and the norms around a block where they are used rather
than where they are computed: streams, graphs, states in place, packed rows,
large offsets, gradients against differences, refusals, and a layer of them
together."""
import numpy as np
import pytest

import oracle.block_oracle as K
import oracle.layer_oracle as L
from tests.test_gpu_block_ops import lin_case
from tests.test_gpu_layer_ops import check, dev_of, dev_spans, round_to, same, seqs_of

pytestmark = pytest.mark.gpu


def ops():
    from gated_delta_rule_recurrence_amd import ops
    return ops


def small_state(dev, dtype="bf16", seed=0, T=150, head=False):
    """Inputs of one small call of each."""
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s: torch.randn(*s, device=dev, generator=g)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    B, Hk, Hv, Dk, Dv, C = 2, 2, 4, 64, 48, 4 * 48
    r = lambda *s: n(*s).to(t)
    lg = -torch.rand(Hv, device=dev, generator=g) if head else -torch.rand(B, T, Hv, device=dev, generator=g)
    return dict(lin=(r(B, T, Hk, Dk), (n(B, T, Hk, Dk) * Dk ** -0.5).to(t), r(B, T, Hv, Dv), lg, n(B, Hv, Dv, Dk)),
                dy=r(B, T, Hv, Dv), dS=n(B, Hv, Dv, Dk),
                res=(r(B, T, C), n(B, T, C), r(B, C), r(C), r(C), r(C), r(C)), dyr=r(B, T, C), dh=n(B, T, C))


HOW = dict(alpha=0.5, center=True)


def run_all(s):
    """Forward and backward of both; every output, in order."""
    y, S_T, saved = ops().gdr_lin_forward(*s["lin"], scale=0.5)
    out = [y, S_T, *ops().gdr_lin_backward(*s["lin"][:4], saved, s["dy"], s["dS"])]
    y, h, stats = ops().gdr_res_forward(*s["res"], **HOW)
    return out + [y, h, stats, *ops().gdr_res_backward(*s["res"], stats, s["dyr"], s["dh"], **HOW)]


@pytest.mark.parametrize("T", (3, 150, 700))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_repeats_are_bitwise_equal(cuda, dtype, T):
    s = small_state(cuda, dtype, T=T, head=T == 150)
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
    import torch
    states = [small_state(cuda, seed=k, T=400) for k in range(2)]
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


@pytest.mark.parametrize("T", (5, 500))
def test_captured_and_replayed(cuda, T):
    """A graph of all calls, replayed on new inputs with eager calls and
    synchronizations between; a second graph of its own beside it."""
    import torch
    states = [small_state(cuda, T=T, seed=k) for k in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_all(states[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in states:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run_all(s))
    flat = lambda d: [t for k in d for t in (d[k] if isinstance(d[k], tuple) else (d[k],))]
    for seed in (3, 4, 5):
        new = [small_state(cuda, T=T, seed=seed + 10 * k) for k in range(2)]
        for s, n in zip(states, new):
            for a, b in zip(flat(s), flat(n)):
                a.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, n in zip(outs, new):
            assert same(out, run_all(n)), seed
        for g in graphs[::-1]:
            g.replay()
        for out, s in zip(outs, states):
            assert same(out, run_all(s)), seed


def test_a_graph_whose_spans_change(cuda):
    """Packed rows in a graph, replayed on other cuts of them (empty
    sequences, gaps, one long one), the states carried in place."""
    import torch
    s = small_state(cuda, seed=4)
    cuts = [[(0, 100), (100, 100), (110, 290)], [(0, 0), (3, 4), (4, 300)], [(290, 300), (300, 300), (300, 300)],
            [(0, 20), (40, 60), (80, 297)]]
    spans = torch.tensor(cuts[0], dtype=torch.int32, device=cuda)
    args = [t.flatten(0, 1) for t in s["lin"][:4]]
    dy = s["dy"].flatten(0, 1)

    def run(S):
        y, S_T, saved = ops().gdr_lin_forward(*args, S, spans=spans, T=300, S_T=S)
        return [y, *ops().gdr_lin_backward(*args, saved, dy, want_dS0=False)[:4]]
    S = torch.zeros(3, 4, 48, 64, device=cuda)
    mine = S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(S)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(S)
    S.zero_()
    for cut in cuts:
        spans.copy_(torch.tensor(cut, dtype=torch.int32, device=cuda))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, run(mine)), cut
        assert torch.equal(S, mine)


@pytest.mark.parametrize("T", (1, 40, 900))
def test_states_in_place(cuda, T):
    import torch
    s = small_state(cuda, T=T)
    y0, S_T, _ = ops().gdr_lin_forward(*s["lin"], save=False)
    for save in (False, True):
        mine = s["lin"][4].clone()
        y1, _, saved = ops().gdr_lin_forward(*s["lin"][:4], mine, save=save, S_T=mine)
        assert torch.equal(y0, y1) and torch.equal(S_T, mine)
    want = ops().gdr_lin_backward(*s["lin"][:4], ops().gdr_lin_forward(*s["lin"])[2], s["dy"])
    assert same(ops().gdr_lin_backward(*s["lin"][:4], saved, s["dy"]), want)  # S0 is in the save buffer


def test_spans_are_cut_to_the_rows(cuda):
    """Spans outside 0 .. rows, and sequences longer than T."""
    import torch
    s = small_state(cuda)
    args = [t.flatten(0, 1) for t in s["lin"][:4]]
    for bad, good, T in (([[-5, 40], [200, 900]], [[0, 40], [200, 300]], 300), ([[0, 100], [150, 90]], [[0, 100], [150, 150]], 300),
                         ([[0, 100], [400, 500]], [[0, 100], [300, 300]], 300), ([[0, 100], [100, 300]], [[0, 70], [100, 170]], 70)):
        out = []
        for c in (bad, good):
            sp = torch.tensor(c, dtype=torch.int32, device=cuda)
            y, S, saved = ops().gdr_lin_forward(*args, s["lin"][4], spans=sp, T=T)
            out.append([y, S, *ops().gdr_lin_backward(*args, saved, s["dy"].flatten(0, 1))])
        assert same(*out), bad


def test_a_longest_length_far_above_the_rows(cuda):
    import torch
    s = small_state(cuda)
    args = [t.flatten(0, 1) for t in s["lin"][:4]]
    sp = torch.tensor([[0, 100], [100, 300]], dtype=torch.int32, device=cuda)
    out = []
    for T in (300, (1 << 30) - 1):
        y, S, saved = ops().gdr_lin_forward(*args, s["lin"][4], spans=sp, T=T)
        out.append([y, S, *ops().gdr_lin_backward(*args, saved, s["dy"].flatten(0, 1))])
    assert same(*out)


def test_no_rows_and_no_sequences(cuda):
    import torch
    s = small_state(cuda)
    q, k, v, lg, S0 = s["lin"]
    none = [t[:, :0] for t in (q, k, v, lg)]
    y, S_T, saved = ops().gdr_lin_forward(*none, S0)
    assert y.shape == (2, 0, 4, 48) and torch.equal(S_T, S0)
    g = ops().gdr_lin_backward(*none, saved, v[:, :0].contiguous(), s["dS"])
    assert torch.equal(g[4], s["dS"]) and g[3].shape == (2, 0, 4)
    y, S_T, saved = ops().gdr_lin_forward(*none[:3], torch.zeros(4, device=cuda), S0)
    g = ops().gdr_lin_backward(*none[:3], torch.zeros(4, device=cuda), saved, v[:, :0].contiguous())
    assert not g[3].any() and not g[4].any()
    none = [t[:0] for t in (q, k, v, lg)]
    y, S_T, saved = ops().gdr_lin_forward(*none)
    assert y.shape == (0, 150, 4, 48) and S_T.shape == (0, 4, 48, 64)
    ops().gdr_lin_backward(*none, saved, v[:0])
    x, r, gate, *w = s["res"]
    y, h, stats = ops().gdr_res_forward(x[:0], r[:0], None, *w, **HOW)
    g = ops().gdr_res_backward(x[:0], r[:0], None, *w, stats, x[:0], r[:0], **HOW)
    assert y.shape == (0, 150, 192) and not any(t.any() for t in g[3:])
    y, h, stats = ops().gdr_res_forward(x[:, :0], r[:, :0], gate, *w, **HOW)
    g = ops().gdr_res_backward(x[:, :0], r[:, :0], gate, *w, stats, x[:, :0].contiguous(), r[:, :0].contiguous(), **HOW)
    assert not g[2].any()


def test_offsets_beyond_32_bits(cuda):
    """Rows whose elements lie past 2^32: the last sequence of a long packed
    buffer, against the same rows in a buffer of their own."""
    import torch
    H, D, R, n = 128, 128, 1 << 18, 90
    g = torch.Generator(device=cuda).manual_seed(3)
    big = torch.empty(R + n, H, D, dtype=torch.bfloat16, device=cuda)
    tail = torch.randn(n, H, D, device=cuda, generator=g).bfloat16()
    big[R:] = tail
    big[5:40] = tail[:35]
    lg = -torch.rand(R + n, H, device=cuda, generator=g)
    both, blg = torch.cat([tail[:35], tail]), torch.cat([lg[5:40], lg[R:]])
    spans = torch.tensor([[5, 40], [R, R + n]], dtype=torch.int32, device=cuda)
    own = torch.tensor([[0, 35], [35, 35 + n]], dtype=torch.int32, device=cuda)
    out = torch.empty_like(big)
    for T in (n, 8):  # tiles, single steps
        _, S_T, _ = ops().gdr_lin_forward(big, big, big, lg, scale=0.01, spans=spans, T=T, save=False, y=out)
        y, S, _ = ops().gdr_lin_forward(both, both, both, blg, scale=0.01, spans=own, T=T, save=False)
        m = min(T, 35)
        assert torch.equal(S_T, S) and torch.equal(out[R:R + T], y[35:35 + T]) and torch.equal(out[5:5 + m], y[:m])
    x = big.view(R + n, H * D)[:, :4096]
    h = torch.empty(R + n, 4096, dtype=torch.bfloat16, device=cuda)
    y, _, _ = ops().gdr_res_forward(x, x, save=False, h=h)
    ty, th, _ = ops().gdr_res_forward(x[R:], x[R:], save=False)
    assert torch.equal(y[R:], ty) and torch.equal(h[R:], th)


def test_gradients_against_differences(cuda):
    """Central differences of the fp32 forward along a random direction v
    against the gradient: (f(x + h v) - f(x - h v)) / 2h against Simpson's mean
    of <grad f, v> over [-h, h], which leaves h^4 / 180 of the fifth derivative.
    At h = 1e-2 the rounding of the difference, 2^-24 |<dy, y>|_1 / h, stays
    below 2e-3 of sum |grad v|."""
    import torch
    s = small_state(cuda, "f32", seed=9)
    gen = torch.Generator(device=cuda).manual_seed(10)
    fs = dict(lin=lambda *a: ops().linear_attention(*a, scale=0.5), res=lambda *a: ops().residual_norm(*a, **HOW))
    dys = dict(lin=(s["dy"], s["dS"]), res=(s["dyr"], s["dh"]))
    h = 1e-2
    for name, f in fs.items():
        args = [t.clone() for t in s[name]]
        for i, t in enumerate(args):
            v = torch.randn(t.shape, device=cuda, generator=gen)
            value, slope, scale = {}, {}, 0.0
            for e in (-h, 0.0, h):
                x = (t + e * v).requires_grad_()
                out = f(*[x if k == i else a for k, a in enumerate(args)])
                value[e] = sum((y.detach().double() * d.double()).sum() for y, d in zip(out, dys[name]))
                torch.autograd.backward(out, dys[name])
                slope[e] = (x.grad.double() * v.double()).sum()
                scale = max(scale, float((x.grad.double() * v.double()).abs().sum()))
            got = (value[h] - value[-h]) / (2 * h)
            want = (slope[-h] + 4 * slope[0.0] + slope[h]) / 6
            assert abs(got - want) <= 2e-3 * scale, (name, i, float(got), float(want), scale)


def test_autograd_of_shared_and_broadcast_inputs(cuda):
    """One tensor as several inputs (its gradients add up), an expanded decay,
    a strided slice, gradients that arrive as views."""
    import torch
    s = small_state(cuda, "f32")
    q, k, v, lg, S0 = s["lin"]
    one = q.clone().requires_grad_()
    ops().linear_attention(one, one, v, lg)[0].backward(s["dy"])
    a, b = q.clone().requires_grad_(), q.clone().requires_grad_()
    ops().linear_attention(a, b, v, lg)[0].backward(s["dy"])
    torch.testing.assert_close(one.grad, a.grad + b.grad, rtol=1e-6, atol=1e-6)
    rate = torch.full((4,), -0.1, device=cuda, requires_grad=True)
    ops().linear_attention(q, k, v, rate.expand(2, 150, 4).contiguous())[0].backward(s["dy"])
    head = torch.full((4,), -0.1, device=cuda, requires_grad=True)
    ops().linear_attention(q, k, v, head)[0].backward(s["dy"])
    torch.testing.assert_close(rate.grad, head.grad, rtol=1e-4, atol=1e-4)
    wide = torch.randn(2, 150, 3 * 128, device=cuda).requires_grad_()
    cut = lambda t: t[..., 128:256].unflatten(-1, (2, 64))
    ops().linear_attention(cut(wide), k, v, lg)[0].backward(s["dy"])
    own = cut(wide.detach()).contiguous().requires_grad_()
    ops().linear_attention(own, k, v, lg)[0].backward(s["dy"])
    assert torch.equal(cut(wide.grad), own.grad) and not wide.grad[..., :128].any()
    x = torch.randn(3, 7, 40, device=cuda)
    both = x.clone().requires_grad_()  # the block's output as its own residual
    y, h = ops().residual_norm(both, both)
    (y + h).sum().backward()
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    y, h = ops().residual_norm(a, b)
    (y + h).sum().backward()
    torch.testing.assert_close(both.grad, a.grad + b.grad, rtol=1e-6, atol=1e-6)
    odd = torch.randn(1 + 3 * 7 * 40, device=cuda)[1:].view(3, 7, 40)
    got = []
    for d in (odd, odd.clone()):
        t = x.clone().requires_grad_()
        y, h = ops().residual_norm(t, x)
        torch.autograd.backward((y, h), (d, d))
        got.append((t.grad,))
    assert same(*got)


def test_only_some_gradients_are_wanted(cuda):
    import torch
    s = small_state(cuda)
    q, k, v, lg, S0 = s["lin"]
    q = q.clone().requires_grad_()
    y, S = ops().linear_attention(q, k, v, lg, S0)
    y.backward(s["dy"])
    assert q.grad is not None and lg.grad is None
    with torch.no_grad():
        y2, S2 = ops().linear_attention(q, k, v, lg, S0)
    assert torch.equal(y, y2) and not y2.requires_grad
    x, r, gate, *w = s["res"]
    r = r.clone().requires_grad_()
    y, h = ops().residual_norm(x, r, gate, *w[:2], pre=False)
    assert y is None
    h.backward(s["dh"])
    assert torch.equal(r.grad, s["dh"])


def test_spans_changed_before_the_backward(cuda):
    import torch
    x = torch.randn(12, 2, 8, device=cuda, requires_grad=True)
    spans = torch.tensor([[0, 12]], dtype=torch.int32, device=cuda)
    y, _ = ops().linear_attention(x, x, x, spans=spans)
    spans[0, 1] = 9
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_refusals(cuda):
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    s = small_state(cuda)
    q, k, v, lg, S0 = s["lin"]
    lin = ops().gdr_lin_forward
    for bad in (lambda: lin(q, k[:, :149], v, lg), lambda: lin(q, k.float(), v, lg), lambda: lin(q, k, v[..., 0, :], lg),
                lambda: lin(q, k, v, lg[..., :3]), lambda: lin(q, k, v, lg.half()), lambda: lin(q, k, v, lg[0, 0, :3]),
                lambda: lin(q, k, v, lg, S0[:1]), lambda: lin(q, k, v, lg, S0.bfloat16()), lambda: lin(q.cpu(), k, v, lg),
                lambda: lin(q, k, v, lg.cpu()), lambda: lin(q.half(), k.half(), v.half(), lg), lambda: lin(q, None, v, lg),
                lambda: lin(q, k, v, 0.5), lambda: lin(q.transpose(0, 1), k, v, lg), lambda: lin(q, k, v, lg, y=q),
                lambda: lin(q, k, v, lg, spans=torch.zeros(2, 2, device=cuda)), lambda: lin(q[..., ::2], k[..., ::2], v, lg),
                lambda: lin(q, k, v, lg, workspace=torch.empty(0, device=cuda), ckpt=torch.empty(4, device=cuda))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(_lib.GdrError, match="multiple"):
        lin(q, k, v[:, :, :3].contiguous(), lg[..., :3].contiguous())
    with pytest.raises(_lib.GdrError, match="256"):
        lin(torch.zeros(1, 2, 1, 257, device=cuda), torch.zeros(1, 2, 1, 257, device=cuda), torch.zeros(1, 2, 1, 4, device=cuda))
    with pytest.raises(_lib.GdrError, match="aligned"):
        lin(q.flatten(2)[..., 1:65].unflatten(-1, (1, 64)), k[:, :, :1].contiguous(), v, lg)
    _, _, saved = lin(q, k, v, lg, S0)
    back = ops().gdr_lin_backward
    for bad in (lambda: back(q, k, v, lg, saved, s["dy"][:, :149]), lambda: back(q, k, v, lg, saved, s["dy"].float()),
                lambda: back(q, k, v, lg, saved, s["dy"], s["dS"][:1])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    saved.ckpt = saved.ckpt[:-1]
    with pytest.raises(ValueError, match="saved.ckpt too small"):
        back(q, k, v, lg, saved, s["dy"])
    x, r, gate, pw, pb, w, b = s["res"]
    res = ops().gdr_res_forward
    for bad in (lambda: res(x, r[:1]), lambda: res(x, r.half()), lambda: res(x, None), lambda: res(x, r, gate[:1]),
                lambda: res(x, r, gate[:, :10]), lambda: res(x, r, None, pw[:5]), lambda: res(x, r, None, pw, pb.float()),
                lambda: res(x, r, None, pw, post=False), lambda: res(x, r, pre_weight=w, pre=False), lambda: res(x[0, 0], r[0, 0]),
                lambda: res(x, r, gate.cpu()), lambda: res(x, r, h=x), lambda: res(x, r, gate[:, None].expand(2, 150, 192))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(_lib.GdrError, match="eps"):
        res(x, r, eps=float("nan"))
    with pytest.raises(_lib.GdrError, match="dimension"):
        res(torch.zeros(1, 8200, device=cuda), torch.zeros(1, 8200, device=cuda))
    with pytest.raises(_lib.GdrError, match="dtype"):
        res(x.float(), r.bfloat16())
    y, h, stats = res(x, r, gate, pw, pb, w, b, center=True)
    back = ops().gdr_res_backward
    for bad in (lambda: back(x, r, gate, pw, pb, w, b, stats, None, s["dh"]), lambda: back(x, r, gate, pw, pb, w, b, None, x),
                lambda: back(x, r, gate, pw, pb, None, None, stats, None, None, pre=False),
                lambda: back(x, r, gate, pw, pb, w, b, stats, s["dyr"], s["dh"].bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_every_call_records_every_event(cuda):
    """The measurement hook, one call at a time."""
    import torch
    from gated_delta_rule_recurrence_amd import _lib
    s = small_state(cuda, T=500)
    lin = [None]

    def forward():
        lin[0] = ops().gdr_lin_forward(*s["lin"])[2]
    stats = ops().gdr_res_forward(*s["res"], **HOW)[2]
    calls = (forward, lambda: ops().gdr_lin_backward(*s["lin"][:4], lin[0], s["dy"]),
             lambda: ops().gdr_res_forward(*s["res"], **HOW),
             lambda: ops().gdr_res_backward(*s["res"], stats, s["dyr"], s["dh"], **HOW))
    for call in calls:
        call()
        events = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
        for e in events:
            e.record()
        mark = torch.cuda.Event(enable_timing=True)
        mark.record()
        torch.cuda.synchronize()
        assert _lib.set_launch_events([e.cuda_event for e in events]) == 0
        try:
            call()
            torch.cuda.synchronize()
        finally:
            assert _lib.set_launch_events([]) == 0
        times = [mark.elapsed_time(e) for e in events]
        assert times == sorted(times) and times[0] > 0


def test_block_together(cuda):
    """Two layers as they stand in a model: the norm before a block, its
    convolution, linear attention, the gated norm of its heads, and the norms
    and the residual sum behind it, which make the next layer's input; one
    training step through autograd against the composed oracles, and the same
    tokens served one by one."""
    import torch

    import oracle.gdr_oracle as O
    B, T, Hk, Hv, Dk, Dv = 2, 90, 2, 4, 16, 24
    nq, nv = Hk * Dk, Hv * Dv
    C = 2 * nq + nv
    r = np.random.default_rng(11)
    f = lambda a: round_to(a, "f32")
    x, w, b = f(r.normal(size=(B, T, C)) * 0.5), f(r.normal(size=(C, 4)) * 0.5), f(r.normal(size=C) * 0.1)
    lg, z = f(-r.exponential(0.2, (B, T, Hv))), f(r.normal(size=(B, T, nv)))
    nw, res = f(1 + 0.1 * r.normal(size=Dv)), f(r.normal(size=(B, T, nv)))
    gate, pw, pre = f(r.normal(size=(B, nv))), f(0.1 * r.normal(size=nv)), f(0.1 * r.normal(size=nv))
    dy, dh = f(r.normal(size=(B, T, nv))), f(r.normal(size=(B, T, nv)))
    leaf = lambda a: dev_of(a, "f32", cuda).requires_grad_()
    X, W, Bi, LG, Z, NW, R, GA, PW, PR = map(leaf, (x, w, b, lg, z, nw, res, gate, pw, pre))
    how = dict(alpha=0.7, weight_offset=1.0)

    def heads(h, n):
        return (h[..., :nq].reshape(B, n, Hk, Dk), h[..., nq:2 * nq].reshape(B, n, Hk, Dk), h[..., 2 * nq:].reshape(B, n, Hv, Dv))
    h, _ = ops().causal_conv(X, W, Bi)
    y, _ = ops().linear_attention(*heads(h, T), LG, scale=0.25)  # slices of one projection, as they are
    o = ops().group_norm(y.reshape(B, T, nv), NW, None, Z, groups=Hv)
    out, stream = ops().residual_norm(o, R, GA, PW, None, PR, **how)
    torch.autograd.backward((out, stream), (dev_of(dy, "f32", cuda), dev_of(dh, "f32", cuda)))

    seqs = seqs_of(B, T, None)
    flat = lambda a: a.reshape(B * T, *a.shape[2:])
    hr, _ = L.conv_forward(flat(x), w, b, None, True, seqs)
    qr, kr, vr = hr[:, :nq].reshape(-1, Hk, Dk), hr[:, nq:2 * nq].reshape(-1, Hk, Dk), hr[:, 2 * nq:].reshape(-1, Hv, Dv)
    yr, _ = K.lin_forward(qr, kr, vr, flat(lg), None, 0.25, seqs)
    orr = L.norm_forward(yr.reshape(-1, nv), nw, None, flat(z), Hv, 1e-6, False, True)
    args = (orr, flat(res), gate, pw, None, pre, None, 0.7, 1e-6, 1, 1, 0)
    outr, streamr = K.res_forward(*args, offset=1.0)
    do, dres, dgate, dpw, _, dpre, _ = K.res_backward(*args, dy=flat(dy), dh=flat(dh), offset=1.0)
    dyr, dwr, _, dzr = L.norm_backward(yr.reshape(-1, nv), nw, None, flat(z), Hv, 1e-6, False, True, do)
    dq, dk, dv, dlg, _ = K.lin_backward(qr, kr, vr, flat(lg), None, 0.25, seqs, dyr.reshape(-1, Hv, Dv), None)
    dhr = np.concatenate([dq.reshape(-1, nq), dk.reshape(-1, nq), dv.reshape(-1, nv)], 1)
    dxr, dcw, dcb, _ = L.conv_backward(flat(x), w, b, None, True, seqs, dhr)
    # each stage's 1e-5 in relative L2, times the condition of the stages
    # before and behind it, at most 10 each
    for name, got, ref in (("out", out, outr), ("stream", stream, streamr), ("dx", X.grad, dxr), ("dw", W.grad, dcw),
                           ("db", Bi.grad, dcb), ("dlg", LG.grad, dlg), ("dz", Z.grad, dzr),
                           ("dnw", NW.grad, dwr.reshape(Hv, Dv).sum(0)), ("dres", R.grad, dres), ("dgate", GA.grad, dgate),
                           ("dpw", PW.grad, dpw), ("dpre", PR.grad, dpre)):
        err = O.rel_l2(got.detach().double().cpu().numpy().reshape(ref.shape), ref)
        assert err <= 1e-4, (name, err)

    with torch.no_grad():  # served: a prompt of 70 tokens, then one by one
        window = state = None
        served = []
        for i, j in [(0, 70)] + [(t, t + 1) for t in range(70, T)]:
            cut = lambda t: t[:, i:j].contiguous()
            h, window = ops().gdr_conv_forward(cut(X), W, Bi, window)
            y, state, _ = ops().gdr_lin_forward(*heads(h, j - i), cut(LG), state, scale=0.25, save=False)
            o, _ = ops().gdr_norm_forward(y.reshape(B, j - i, nv), NW, None, cut(Z), groups=Hv, save=False)
            p, _, _ = ops().gdr_res_forward(o, cut(R), GA, PW, None, PR, save=False, **how)
            served.append(p)
    err = O.rel_l2(torch.cat(served, 1).double().cpu().numpy().reshape(outr.shape), outr)
    assert err <= 1e-4, err


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("spans,rows", (
    ([(0, 1200), (0, 0), (500, 500), (1203, 1290), (1300, 1300), (7, 7)], 1300),  # cut and joined
    ([(0, 0), (2, 50), (50, 50), (0, 0), (60, 120), (0, 0)], 120),                # one piece each
    ([(9, 9), (0, 6), (0, 0), (6, 7), (10, 10), (7, 10), (3, 3)], 10)))           # step by step
def test_empty_sequences_anywhere(cuda, dtype, spans, rows):
    """Sequences of no rows whose spans point into others' rows: they keep
    their states and leave what the others save alone."""
    lin_case(cuda, dtype, len(spans), 0, 1, 2, 64, 64, spans=spans, rows=rows, rate=0.02)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("T", (100, 300))
@pytest.mark.parametrize("what", (float("nan"), float("inf"), float("-inf")))
def test_not_finite_rows(cuda, dtype, T, what):
    """A value that is not finite reaches the outputs that depend on it, and no
    other: not the earlier steps of its tile, its neighbouring columns or other
    heads; the gradients likewise."""
    import torch
    s = small_state(cuda, dtype, T=T)
    q, k, v, lg, S0 = s["lin"]
    at, h, c = 70, 1, 5
    run = lambda *a: ops().gdr_lin_forward(*a, S0, scale=0.5)
    y, S, saved = run(q, k, v, lg)
    grads = ops().gdr_lin_backward(q, k, v, lg, saved, s["dy"], s["dS"])

    def poison(t, head):
        t = t.clone()
        t[0, at, head, c] = what
        return t

    y2, S2, _ = run(q, k, poison(v, h), lg)  # one column of one value head
    reached = torch.zeros_like(y, dtype=torch.bool)
    reached[0, at:, h, c] = True
    assert torch.equal(y2[~reached], y[~reached]) and not torch.isfinite(y2[reached]).any()
    reached = torch.zeros_like(S, dtype=torch.bool)
    reached[0, h, c] = True
    assert torch.equal(S2[~reached], S[~reached]) and not torch.isfinite(S2[reached]).any()
    y2, S2, _ = run(q, poison(k, 0), v, lg)  # key head 0: value heads 0 and 1
    assert torch.equal(y2[0, :at], y[0, :at]) and torch.equal(y2[:, :, 2:], y[:, :, 2:]) and torch.equal(y2[1], y[1])
    assert not torch.isfinite(y2[0, at:, :2]).any()
    y2, S2, _ = run(poison(q, 0), k, v, lg)
    reached = torch.zeros_like(y, dtype=torch.bool)
    reached[0, at, :2] = True
    assert torch.equal(y2[~reached], y[~reached]) and torch.equal(S2, S) and not torch.isfinite(y2[reached]).any()
    # dy: dq of its row, dk and dv of its own and earlier ones
    dq, dk, dv, _, dS0 = ops().gdr_lin_backward(q, k, v, lg, saved, poison(s["dy"], h), s["dS"])
    for got, want, rows, heads in ((dq, grads[0], slice(at, at + 1), slice(0, 1)), (dk, grads[1], slice(0, at + 1), slice(0, 1)),
                                   (dv, grads[2], slice(0, at + 1), slice(h, h + 1))):
        reached = torch.zeros_like(got, dtype=torch.bool)
        reached[0, rows, heads, c if got is dv else slice(None)] = True
        assert torch.equal(got[~reached], want[~reached]) and not torch.isfinite(got[reached]).any()
    reached = torch.zeros_like(dS0, dtype=torch.bool)
    reached[0, h, c] = True
    assert torch.equal(dS0[~reached], grads[4][~reached]) and not torch.isfinite(dS0[reached]).any()
