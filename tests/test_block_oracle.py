"""CPU pins of the float64 definitions of linear attention and of the norms
around a block: identities, other forms of the same sums, and differences."""
import numpy as np
import pytest

import oracle.block_oracle as L


def lin_inputs(seed=0, rows=23, Hk=2, Hv=4, Dk=5, Dv=3, B=3):
    r = np.random.default_rng(seed)
    q, k, v = r.normal(size=(rows, Hk, Dk)), r.normal(size=(rows, Hk, Dk)), r.normal(size=(rows, Hv, Dv))
    return q, k, v, -r.exponential(0.4, size=(rows, Hv)), r.normal(size=(B, Hv, Dv, Dk))


SEQS = [(0, 7), (7, 7), (9, 22)]


def test_lin_forward_is_the_sum_over_earlier_steps():
    q, k, v, lg, S0 = lin_inputs()
    y, S_T = L.lin_forward(q, k, v, lg, S0, 0.7, SEQS)
    for b, (i, j) in enumerate(SEQS):
        for h in range(4):
            G = np.cumsum(lg[i:j, h])
            S = S0[b, h]
            for t in range(i, j):
                want = np.exp(G[t - i]) * S0[b, h] @ q[t, h // 2]
                for m in range(i, t + 1):
                    want = want + np.exp(G[t - i] - G[m - i]) * (k[m, h // 2] @ q[t, h // 2]) * v[m, h]
                np.testing.assert_allclose(y[t, h], 0.7 * want, rtol=1e-11, atol=1e-12)
                S = np.exp(lg[t, h]) * S + np.outer(v[t, h], k[t, h // 2])
            np.testing.assert_allclose(S_T[b, h], S, rtol=1e-12)
    assert not y[7:9].any() and not y[22:].any()
    np.testing.assert_array_equal(S_T[1], S0[1])  # no rows: the state stays


def test_lin_without_decay_and_with_one_per_head():
    q, k, v, lg, S0 = lin_inputs(1)
    whole = [(0, 23)]
    y, S = L.lin_forward(q, k, v, None, None, 1.0, whole)
    np.testing.assert_allclose(S[0, 3], v[:, 3].T @ k[:, 1], rtol=1e-12)
    head = lg[0]
    a = L.lin_forward(q, k, v, head, S0[:1], 1.0, whole)
    b = L.lin_forward(q, k, v, np.repeat(head[None], 23, 0), S0[:1], 1.0, whole)
    for x, z in zip(a, b):
        np.testing.assert_array_equal(x, z)


def test_lin_is_the_gated_delta_rule_without_its_correction():
    """beta_t = 1 and keys orthogonal to every earlier one leave no correction."""
    import oracle.gdr_oracle as O
    r = np.random.default_rng(2)
    T, H, D = 6, 2, 6
    k = np.stack([np.linalg.qr(r.normal(size=(D, D)))[0].T for _ in range(H)], 1)  # [T, H, D]
    q, v = r.normal(size=(T, H, D)), r.normal(size=(T, H, 4))
    lg = -r.exponential(0.3, size=(T, H))
    y, S = O.forward(q[None], k[None], v[None], np.exp(lg)[None], np.ones((1, T, H)), None)
    z, Z = L.lin_forward(q, k, v, lg, None, 1.0, [(0, T)])
    np.testing.assert_allclose(z, y[0], rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(Z[0], S[0], rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("head", (False, True))
def test_lin_backward_against_differences(head):
    q, k, v, lg, S0 = lin_inputs(3)
    lg = lg[0] if head else lg
    r = np.random.default_rng(4)
    dy, dS = r.normal(size=v.shape), r.normal(size=S0.shape)
    args = [q, k, v, lg, S0]
    grads = L.lin_backward(*args, 0.7, SEQS, dy, dS)

    def loss(a):
        y, S = L.lin_forward(*a, 0.7, SEQS)
        return (y * dy).sum() + (S * dS).sum()
    for n, g in zip(range(5), grads):
        for _ in range(6):
            at = tuple(r.integers(0, s) for s in args[n].shape)
            moved = []
            for e in (1e-5, -1e-5):
                a = [x.copy() for x in args]
                a[n][at] += e
                moved.append(loss(a))
            np.testing.assert_allclose(g[at], (moved[0] - moved[1]) / 2e-5, rtol=1e-6, atol=1e-7)


def test_lin_decay_gradient_is_what_enters_less_what_leaves():
    """Behind step t: the queries' share of the states from before them, less
    the keys' share of the states behind them, and the last state's."""
    q, k, v, lg, S0 = lin_inputs(5)
    r = np.random.default_rng(6)
    dy, dS = r.normal(size=v.shape), r.normal(size=S0.shape)
    dg = L.lin_backward(q, k, v, lg, S0, 0.7, SEQS, dy, dS)[3]
    _, S_T = L.lin_forward(q, k, v, lg, S0, 0.7, SEQS)
    one = lambda x: np.repeat(x, 2, 1)
    heads = L.lin_backward(one(q), one(k), v, lg, S0, 0.7, SEQS, dy, dS)  # dq, dk of each value head
    flow = (one(q) * heads[0]).sum(2) - (one(k) * heads[1]).sum(2)
    for b, (i, j) in enumerate(SEQS):
        end = (dS[b] * S_T[b]).sum((1, 2))
        want = flow[i:j][::-1].cumsum(0)[::-1] + end
        np.testing.assert_allclose(dg[i:j], want, rtol=1e-8, atol=1e-9)


def res_inputs(seed, n, rows=6, C=7):
    r = np.random.default_rng(seed)
    z = lambda *s: r.normal(size=s)
    return z(rows, C), z(rows, C), None if n == 0 else z(n, C), 1 + 0.2 * z(C), z(C), 1 + 0.2 * z(C), z(C)


@pytest.mark.parametrize("n", (0, 1, 2, 6))
@pytest.mark.parametrize("post,pre,center,offset", ((1, 1, 0, 0.0), (0, 1, 1, 1.0), (1, 0, 1, 0.0), (1, 1, 1, 1.0)))
def test_res_backward_against_differences(n, post, pre, center, offset):
    args = list(res_inputs(n, n))
    r = np.random.default_rng(8)
    dy, dh = r.normal(size=args[0].shape), r.normal(size=args[0].shape)
    how = dict(alpha=0.6, eps=1e-3, post=post, pre=pre, center=center, offset=offset)
    grads = L.res_backward(*args, dy=dy, dh=dh, **how)

    def loss(a):
        y, h = L.res_forward(*a, **how)
        return (0.0 if y is None else (y * dy).sum()) + (h * dh).sum()
    for i, g in enumerate(grads):
        used = (True, True, n > 0, post, post, pre, pre)[i]
        if not used:
            assert g is None
            continue
        for _ in range(5):
            at = tuple(r.integers(0, s) for s in args[i].shape)
            moved = []
            for e in (1e-5, -1e-5):
                a = [None if x is None else x.copy() for x in args]
                a[i][at] += e
                moved.append(loss(a))
            np.testing.assert_allclose(g[at], (moved[0] - moved[1]) / 2e-5, rtol=1e-5, atol=1e-7)


def test_res_forward_one_row_by_hand():
    x, res = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    y, h = L.res_forward(x, res, np.array([[2.0, 0.5]]), None, None, None, None, 0.1, 0.0, 1, 1, 0)
    n = x / np.sqrt(12.5)
    want = res + 0.1 * np.array([[2.0, 0.5]]) * n
    np.testing.assert_allclose(h, want)
    np.testing.assert_allclose(y, want / np.sqrt((want ** 2).mean()))
    y, h = L.res_forward(x, res, None, None, None, None, None, 1.0, 0.0, 0, 1, 1)
    np.testing.assert_allclose(h, [[4.0, 3.0]])
    np.testing.assert_allclose(y, [[1.0, -1.0]])


def test_magnitudes_bound_the_values():
    q, k, v, lg, S0 = lin_inputs(9)
    r = np.random.default_rng(10)
    dy, dS = r.normal(size=v.shape), r.normal(size=S0.shape)
    for a, b in zip(L.lin_forward(q, k, v, lg, S0, 0.7, SEQS) + L.lin_backward(q, k, v, lg, S0, 0.7, SEQS, dy, dS),
                    L.lin_forward(q, k, v, lg, S0, 0.7, SEQS, mag=True)
                    + L.lin_backward(q, k, v, lg, S0, 0.7, SEQS, dy, dS, mag=True)):
        assert (np.abs(a) <= b + 1e-12).all()
    args = res_inputs(11, 2)
    dy, dh = r.normal(size=args[0].shape), r.normal(size=args[0].shape)
    how = dict(alpha=-0.6, eps=1e-3, post=1, pre=1, center=1, offset=1.0)
    for a, b in zip(L.res_forward(*args, **how) + L.res_backward(*args, dy=dy, dh=dh, **how),
                    L.res_forward(*args, mag=True, **how) + L.res_backward(*args, dy=dy, dh=dh, mag=True, **how)):
        assert (np.abs(a) <= b + 1e-12).all()
