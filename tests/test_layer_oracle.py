"""CPU pins of the layer operators' float64 oracle: every gradient against
central differences, closed forms, and the sequence rules (spans, carried
states) against running the pieces alone."""
import numpy as np
import pytest

import oracle.layer_oracle as L

H = 1e-6


def differences(f, args, which, cot):
    """d <cot, f(args)> / d args[which] by central differences."""
    a = args[which]
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + H
        up = sum((c * o).sum() for c, o in zip(cot, f(*args)))
        a[i] = keep - H
        down = sum((c * o).sum() for c, o in zip(cot, f(*args)))
        a[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


def close(a, b):
    # differences of O(1) values at H = 1e-6 in float64: 1e-16 / 1e-6 of
    # rounding times the number of terms, and H^2 of truncation
    np.testing.assert_allclose(a, b, rtol=2e-6, atol=2e-7)


SEQS = [(0, 3), (3, 3), (4, 5), (5, 9)]  # an empty one, a gap, one of one row
ROWS = 10


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_gradients(act, K):
    r = np.random.default_rng(K)
    C = 3
    x, w, b = r.normal(size=(ROWS, C)), r.normal(size=(C, K)), r.normal(size=C)
    st = r.normal(size=(4, K - 1, C))
    f = lambda *a: L.conv_forward(*a, act, SEQS)
    cot = [r.normal(size=(ROWS, C)), r.normal(size=st.shape)]
    got = L.conv_backward(x, w, b, st, act, SEQS, *cot)
    for k in range(4):
        if st.size or k < 3:
            close(got[k], differences(f, [x, w, b, st], k, cot))


@pytest.mark.parametrize("plus,gated", [(True, True), (False, False), (True, False)])
def test_scan_gradients(plus, gated):
    r = np.random.default_rng(7)
    C, N, G = 4, 3, 2
    n = lambda *s: r.normal(size=s)
    u, dt, z = n(ROWS, C), n(ROWS, C), n(ROWS, C)
    if not plus:
        dt = np.abs(dt) * 0.3
    A, Bm, Cm, D, bias, S0 = -np.exp(n(C, N)), n(ROWS, G, N), n(ROWS, G, N), n(C), n(C) * 0.1, n(4, C, N)
    args = [u, dt, A, Bm, Cm, D, z if gated else None, bias, S0]
    f = lambda *a: L.scan_forward(*a, plus, SEQS)
    cot = [n(ROWS, C), n(4, C, N)]
    got = L.scan_backward(*args, plus, SEQS, *cot)
    for k, name in enumerate(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")):
        if args[k] is not None:
            close(got[name], differences(f, args, k, cot))


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_gradients(center, act, gated, shared):
    r = np.random.default_rng(3)
    R, G, D = 4, 3, 5
    n = lambda *s: r.normal(size=s)
    x, z = n(R, G * D), n(R, G * D) if gated else None
    w, b = n(D if shared else G * D), n(D if shared else G * D)
    f = lambda *a: [L.norm_forward(*a, G, 1e-3, center, act)]
    cot = [n(R, G * D)]
    got = list(L.norm_backward(x, w, b, z, G, 1e-3, center, act, cot[0]))
    if shared:
        got[1], got[2] = (g.reshape(G, D).sum(0) for g in got[1:3])
    for k in range(4):
        if k < 3 or gated:
            close(got[k], differences(f, [x, w, b, z], k, cot))


def test_conv_matches_its_definition_by_hand():
    x = np.arange(1.0, 5.0)[:, None]
    w = np.array([[1.0, 10.0, 100.0]])
    y, st = L.conv_forward(x, w, np.array([0.5]), None, False, [(0, 4)])
    np.testing.assert_array_equal(y[:, 0], [100.5, 210.5, 321.5, 432.5])
    np.testing.assert_array_equal(st[0, :, 0], [3.0, 4.0])


def test_scan_matches_its_definition_by_hand():
    # one channel, one state, delta = 1, exp(A) = 1/2
    one = np.ones((3, 1))
    u = np.array([[1.0], [2.0], [4.0]])
    y, S = L.scan_forward(u, one, np.log(np.array([[0.5]])), one[:, None], 2 * one[:, None], np.array([3.0]),
                          None, None, np.array([[[8.0]]]), False, [(0, 3)])
    # h: 5, 4.5, 6.25
    np.testing.assert_allclose(y[:, 0], [13.0, 15.0, 24.5], rtol=1e-15)
    np.testing.assert_allclose(S, [[[6.25]]], rtol=1e-15)


def test_pieces_carry_the_state():
    r = np.random.default_rng(5)
    n = lambda *s: r.normal(size=s)
    C, N, K = 4, 3, 4
    u, dt, z, A, Bm, Cm, D = n(9, C), n(9, C), n(9, C), -np.exp(n(C, N)), n(9, 2, N), n(9, 2, N), n(C)
    y, S = L.scan_forward(u, dt, A, Bm, Cm, D, z, None, None, True, [(0, 9)])
    y0, S0 = L.scan_forward(u[:4], dt[:4], A, Bm[:4], Cm[:4], D, z[:4], None, None, True, [(0, 4)])
    y1, S1 = L.scan_forward(u[4:], dt[4:], A, Bm[4:], Cm[4:], D, z[4:], None, S0, True, [(0, 5)])
    np.testing.assert_allclose(np.concatenate([y0, y1]), y, rtol=1e-12)
    np.testing.assert_allclose(S1, S, rtol=1e-12)
    w = n(C, K)
    y, s = L.conv_forward(u, w, None, None, True, [(0, 9)])
    y0, s0 = L.conv_forward(u[:2], w, None, None, True, [(0, 2)])
    y1, s1 = L.conv_forward(u[2:], w, None, s0, True, [(0, 7)])
    np.testing.assert_allclose(np.concatenate([y0, y1]), y, rtol=1e-12)
    np.testing.assert_array_equal(s1, s)


def test_magnitudes_bound_the_values():
    """mag=True is at least the value itself, element by element."""
    r = np.random.default_rng(9)
    n = lambda *s: r.normal(size=s)
    C, N, G = 4, 3, 2
    args = [n(ROWS, C), n(ROWS, C), -np.exp(n(C, N)), n(ROWS, G, N), n(ROWS, G, N), n(C), n(ROWS, C), n(C),
            n(4, C, N)]
    cot = [n(ROWS, C), n(4, C, N)]
    for a, m in zip(L.scan_forward(*args, True, SEQS), L.scan_forward(*args, True, SEQS, mag=True)):
        assert (np.abs(a) <= m + 1e-12).all()
    a, m = (L.scan_backward(*args, True, SEQS, *cot, mag=k) for k in (False, True))
    for k in a:
        assert (np.abs(a[k]) <= m[k] + 1e-12).all(), k
    x, w, b, st = n(ROWS, C), n(C, 3), n(C), n(4, 2, C)
    for f in (lambda k: L.conv_forward(x, w, b, st, True, SEQS, mag=k),
              lambda k: L.conv_backward(x, w, b, st, True, SEQS, x, st, mag=k),
              lambda k: L.norm_backward(x, n(4) * 0 + 2, b, n(ROWS, C) * 0 + 1, 2, 1e-3, True, True, x, mag=k)):
        for a, m in zip(f(False), f(True)):
            assert (np.abs(a) <= m + 1e-12).all()
