"""Float64 definitions of linear attention with a decay for each head and of
the norms around a block, each forward and backward.

Test infrastructure only; no code shared with the HIP path.  Rows are flat
[rows, ...]; `seqs` lists each sequence's (first row, row past its last).
Rows of no sequence come out as zeros.

mag=True returns, for every output, the sum of the absolute values of the
terms that make it up (signs dropped in every product, decays, gates' signs
and the norms' statistics kept): an fp32 evaluation that rounds n times on the
way differs from the exact value by at most n 2^-24 times that.
"""
import numpy as np


def _absall(mag, *arrays):
    return [None if a is None else (np.abs(a) if mag else a) for a in arrays]


# ---- linear attention ----------------------------------------------------------

def _decays(log_g, rows, Hv):
    if log_g is None:
        return np.ones((rows, Hv))
    return np.broadcast_to(np.exp(log_g), (rows, Hv))


def lin_forward(q, k, v, log_g, S0, scale, seqs, mag=False):
    """(y, S_T): q, k [rows, Hk, Dk]; v [rows, Hv, Dv]; log_g [rows, Hv], [Hv] or None."""
    rows, Hv, Dv = v.shape
    reps = Hv // q.shape[1]
    g = _decays(log_g, rows, Hv)
    q, k, v, S0 = _absall(mag, q, k, v, S0)
    q, k = np.repeat(q, reps, 1), np.repeat(k, reps, 1)
    y = np.zeros_like(v)
    ends = np.zeros((len(seqs), Hv, Dv, q.shape[2]))
    for b, (i, j) in enumerate(seqs):
        S = ends[b] if S0 is None else S0[b].copy()
        for t in range(i, j):
            S = g[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            y[t] = (abs(scale) if mag else scale) * np.einsum("hvk,hk->hv", S, q[t])
        ends[b] = S
    return y, ends


def lin_backward(q, k, v, log_g, S0, scale, seqs, dy, dS_T, mag=False):
    """(dq, dk, dv, dlog_g, dS0); dlog_g of log_g's shape.  With mag, dlog_g's
    is the sum over later steps of what enters and leaves the states there:
    the terms of the suffix sums that it is formed by."""
    rows, Hv, Dv = v.shape
    Hk, Dk = q.shape[1:]
    reps = Hv // Hk
    g = _decays(log_g, rows, Hv)
    q, k, v, S0, dy, dS_T = _absall(mag, q, k, v, S0, dy, dS_T)
    scale = abs(scale) if mag else scale
    q, k = np.repeat(q, reps, 1), np.repeat(k, reps, 1)
    dq, dk, dv = np.zeros((rows, Hv, Dk)), np.zeros((rows, Hv, Dk)), np.zeros_like(v)
    dg = np.zeros((rows, Hv))
    dS0 = np.zeros((len(seqs), Hv, Dv, Dk))
    for b, (i, j) in enumerate(seqs):
        S = np.zeros((Hv, Dv, Dk)) if S0 is None else S0[b]
        states = []
        for t in range(i, j):
            states.append(S)
            S = g[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            dq[t] = scale * np.einsum("hvk,hv->hk", S, dy[t])
        D = np.zeros((Hv, Dv, Dk)) if dS_T is None else dS_T[b]
        flow = (D * S).sum((1, 2))
        for t in range(j - 1, i - 1, -1):
            leaves = np.einsum("hvk,hv,hk->h", D, v[t], k[t])  # the later steps' part of dk_t k_t
            D = D + scale * dy[t][:, :, None] * q[t][:, None, :]
            dk[t] = np.einsum("hvk,hv->hk", D, v[t])
            dv[t] = np.einsum("hvk,hk->hv", D, k[t])
            before = g[t][:, None, None] * states.pop()
            if mag:
                enters = scale * np.einsum("hvk,hv,hk->h", before, dy[t], q[t])
                flow = flow + enters + leaves
                dg[t] = flow
            else:
                dg[t] = (D * before).sum((1, 2))
            D = g[t][:, None, None] * D
        dS0[b] = D
    shared = lambda x: x.reshape(rows, Hk, reps, Dk).sum(2)
    if log_g is None:
        dg = None
    elif log_g.ndim == 1:
        dg = dg.sum(0)
    return shared(dq), shared(dk), dv, dg, dS0


# ---- the norms around a block ---------------------------------------------------

def _norm(a, w, b, eps, center, offset, mag):
    """(normed, mu, r, xh); with mag the magnitudes of the first and the last,
    for the statistics of a itself."""
    mu = a.mean(1, keepdims=True) if center else np.zeros((len(a), 1))
    r = 1.0 / np.sqrt(((a - mu) ** 2).mean(1, keepdims=True) + eps)
    xh = (a - mu) * r
    if mag:
        # the subtraction loses 2^-24 (|a| + |mu|), the mean up to mean |a|
        xh = (np.abs(a) + (np.abs(a).mean(1, keepdims=True) if center else 0.0)) * r
    w = np.ones(a.shape[1]) if w is None else w + offset
    b = np.zeros(a.shape[1]) if b is None else b
    w, b = _absall(mag, w, b)
    return xh * w + b, mu, r, xh


def _gates(gate, rows, C):
    """gate [n][C], each row serving rows / n rows."""
    if gate is None:
        return np.ones((rows, C))
    g = gate.reshape(-1, C)
    return np.repeat(g, rows // len(g), 0) if rows else np.zeros((0, C))


def res_forward(x, res, gate, pw, pb, w, b, alpha, eps, post, pre, center, offset=0.0, mag=False):
    """(y or None, h) of rows [rows, C]."""
    g = _gates(gate, *x.shape) * alpha
    n = _norm(x, pw, pb, eps, center, offset, False)[0] if post else x
    h = res + g * n
    if not mag:
        return (_norm(h, w, b, eps, center, offset, False)[0] if pre else None), h
    nm = _norm(x, pw, pb, eps, center, offset, True)[0] if post else np.abs(x)
    hm = np.abs(res) + np.abs(g) * nm
    if not pre:
        return None, hm
    # an error of h goes through the norm's slope, r (w + offset), and through its statistics
    mu, r = _norm(h, w, b, eps, center, offset, False)[1:3]
    wm = np.ones(x.shape[1]) if w is None else np.abs(w + offset)
    xh = np.abs(h - mu) * r
    spread = hm * r + hm.mean(1, keepdims=True) * r + xh * (xh * hm * r).mean(1, keepdims=True)
    return _norm(h, w, b, eps, center, offset, True)[0] + spread * wm, hm


def _back(e, xh, r, center, mag):
    s = 1.0 if mag else -1.0
    return r * (e + s * (e.mean(1, keepdims=True) if center else 0.0) + s * xh * (e * xh).mean(1, keepdims=True))


def res_backward(x, res, gate, pw, pb, w, b, alpha, eps, post, pre, center, dy, dh, offset=0.0, mag=False):
    """(dx, dres, dgate, dpw, dpb, dw, db); dgate [n][C]; None where there is
    no such input (dpb, db always formed)."""
    rows, C = x.shape
    g = _gates(gate, rows, C) * alpha
    n, mu1, r1, xh = _norm(x, pw, pb, eps, center, offset, False) if post else (x, None, None, None)
    h = res + g * n
    if mag:
        if post:
            n, _, _, xh = _norm(x, pw, pb, eps, center, offset, True)
        n, g = np.abs(n), np.abs(g)
        hm = np.abs(res) + g * n
    d = np.zeros_like(x) if dh is None else dh
    d, dy = _absall(mag, d, dy)
    wf = np.ones(C) if w is None else w + offset
    pf = np.ones(C) if pw is None else pw + offset
    wf, pf = _absall(mag, wf, pf)
    dw = db = dpw = dpb = None
    if pre:
        _, mu2, r2, hh = _norm(h, w, b, eps, center, offset, False)
        if mag:  # of hh: as y in res_forward
            ah = np.abs(hh)
            hh = (hm + (hm.mean(1, keepdims=True) if center else 0.0)) * r2
            hh = hh + ah * (ah * hm * r2).mean(1, keepdims=True)
        dw, db = (dy * hh).sum(0), dy.sum(0)
        d = d + _back(dy * wf, hh, r2, center, mag)
    dgate = None
    if gate is not None:
        k = gate.size // C
        dgate = (abs(alpha) if mag else alpha) * (d * n).reshape(k, rows // k, C).sum(1) if rows else np.zeros((k, C))
    dn = g * d
    dx = dn
    if post:
        dpw, dpb = (dn * xh).sum(0), dn.sum(0)
        dx = _back(dn * pf, xh, r1, center, mag)
    return dx, d, dgate, dpw, dpb, dw, db
