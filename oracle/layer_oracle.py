"""Float64 definitions of the operators around the recurrence: the short
causal convolution, the selective state space scan and the group norm, each
forward and backward, one step at a time.

Test infrastructure only; no code shared with the HIP path.  Rows are flat
[rows, ...]; `seqs` lists each sequence's (first row, row past its last).
Rows of no sequence come out as zeros.

mag=True returns, for every output, the sum of the absolute values of the
terms that make it up (signs dropped in every product, decays and
activations kept as they are): an fp32 evaluation that rounds n times on the
way differs from the exact value by at most n 2^-24 times that.
"""
import numpy as np


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    return np.logaddexp(0.0, x)


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    return s + x * s * (1.0 - s)


def _absall(mag, *arrays):
    return [None if a is None else (np.abs(a) if mag else a) for a in arrays]


# ---- short causal convolution ------------------------------------------------

def _pre(x, w, bias, state, seqs, mag):
    K = w.shape[1]
    x, w, bias, state = _absall(mag, x, w, bias, state)
    s = np.zeros_like(x)
    full = []
    for b, (i, j) in enumerate(seqs):
        head = np.zeros((K - 1, x.shape[1])) if state is None else state[b]
        f = np.concatenate([head, x[i:j]])
        full.append(f)
        for t in range(j - i):
            s[i + t] = (f[t:t + K] * w.T).sum(0) + (0.0 if bias is None else bias)
    return s, full


def conv_forward(x, w, bias, state, act, seqs, mag=False):
    """(y, state_out)"""
    K = w.shape[1]
    s, full = _pre(x, w, bias, state, seqs, mag)
    out = np.stack([f[len(f) - (K - 1):] for f in full]) if seqs else np.zeros((0, K - 1, x.shape[1]))
    if mag:
        # |act'| <= 1.1; act itself loses about |s| + 4 units of |act(s)|
        return 1.1 * s + 1e-30, np.abs(out)
    y = np.zeros_like(s)
    for i, j in seqs:
        y[i:j] = silu(s[i:j]) if act else s[i:j]
    return y, out


def conv_backward(x, w, bias, state, act, seqs, dy, dstate_out=None, mag=False):
    """(dx, dw, dbias, dstate)"""
    K = w.shape[1]
    s, _ = _pre(x, w, bias, state, seqs, False)
    d = np.zeros_like(x)
    for i, j in seqs:
        g = dsilu(s[i:j]) if act else np.ones_like(s[i:j])
        if mag:
            # act' is off by at most |act''| <= 0.5 times the error of s
            sm, _ = _pre(x, w, bias, state, seqs, True)
            g = np.abs(g) + (0.5 * sm[i:j] if act else 0.0)
        d[i:j] = dy[i:j] * g
    x, w, state, d, dso = _absall(mag, x, w, state, d, dstate_out)
    dx, dw, db = np.zeros_like(x), np.zeros_like(w), np.zeros(x.shape[1])
    dst = np.zeros((len(seqs), K - 1, x.shape[1]))
    for b, (i, j) in enumerate(seqs):
        head = np.zeros((K - 1, x.shape[1])) if state is None else state[b]
        f = np.concatenate([head, x[i:j]])
        df = np.zeros_like(f)
        for t in range(j - i):
            df[t:t + K] += d[i + t] * w.T
            dw += (d[i + t] * f[t:t + K]).T
            db += d[i + t]
        if dso is not None:
            df[len(f) - (K - 1):] += dso[b]
        dx[i:j] = df[K - 1:]
        dst[b] = df[:K - 1]
    return dx, dw, db, dst


# ---- selective state space scan ------------------------------------------------

def _steps(dt, dt_bias, plus):
    raw = dt if dt_bias is None else dt + dt_bias
    return raw, (softplus(raw) if plus else raw)


def scan_forward(u, dt, A, Bm, Cm, D, z, dt_bias, S0, plus, seqs, mag=False, history=False):
    """(y, S_T[, states before every row])"""
    C, N = A.shape
    G = Bm.shape[1]
    _, delta = _steps(dt, dt_bias, plus)
    decay = lambda t: np.exp(delta[t][:, None] * A)
    gate = np.ones_like(u) if z is None else silu(z)
    size = np.abs(delta) if mag else delta
    u, Bm, Cm, D, S0, gate = _absall(mag, u, Bm, Cm, D, S0, gate)
    y = np.zeros_like(u)
    S_T = np.zeros((len(seqs), C, N))
    hist = np.zeros((u.shape[0], C, N)) if history else None
    spread = lambda t, m: np.repeat(m[t], C // G, axis=0)  # [C][N]
    for b, (i, j) in enumerate(seqs):
        h = np.zeros((C, N)) if S0 is None else S0[b].copy()
        for t in range(i, j):
            if history:
                hist[t] = h
            h = decay(t) * h + (size[t] * u[t])[:, None] * spread(t, Bm)
            y[t] = ((h * spread(t, Cm)).sum(1) + (0.0 if D is None else D * u[t])) * gate[t]
        S_T[b] = h
    return (y, S_T, hist) if history else (y, S_T)


def scan_backward(u, dt, A, Bm, Cm, D, z, dt_bias, S0, plus, seqs, dy, dS_T=None, mag=False):
    """dict of du, ddt, dA, dB, dC, dD, dz, ddt_bias, dS0"""
    C, N = A.shape
    G = Bm.shape[1]
    raw, delta = _steps(dt, dt_bias, plus)
    decays = [np.exp(delta[t][:, None] * A) for t in range(u.shape[0])]
    hist = scan_forward(u, dt, A, Bm, Cm, D, z, dt_bias, S0, plus, seqs, mag, history=True)[2]
    slope = sigmoid(raw) if plus else np.ones_like(raw)
    g = np.ones_like(u) if z is None else silu(z)
    dg = np.zeros_like(u) if z is None else dsilu(z)
    if mag and z is not None:
        dg = np.abs(dg) + 0.5 * np.abs(z)
    u, Bm, Cm, D, delta, A, g, dg, dy, dS_T = _absall(mag, u, Bm, Cm, D, delta, A, g, dg, dy, dS_T)
    o = dict(du=np.zeros_like(u), ddt=np.zeros_like(u), dA=np.zeros((C, N)), dB=np.zeros_like(Bm),
             dC=np.zeros_like(Cm), dD=np.zeros(C), dz=np.zeros_like(u), ddt_bias=np.zeros(C),
             dS0=np.zeros((len(seqs), C, N)))
    spread = lambda t, m: np.repeat(m[t], C // G, axis=0)
    gather = lambda m: m.reshape(G, C // G, N).sum(1)
    Dv = np.zeros(C) if D is None else D
    for b, (i, j) in enumerate(seqs):
        carry = np.zeros((C, N)) if dS_T is None else dS_T[b].copy()
        for t in range(j - 1, i - 1, -1):
            a, Bt, Ct = decays[t], spread(t, Bm), spread(t, Cm)
            du_in = delta[t] * u[t]
            h = a * hist[t] + du_in[:, None] * Bt
            read = (h * Ct).sum(1) + Dv * u[t]
            out = dy[t] * g[t]
            o["dz"][t] = dy[t] * read * dg[t]
            e = carry + out[:, None] * Ct
            o["dC"][t] = gather(out[:, None] * h)
            o["dB"][t] = gather(e * du_in[:, None])
            eB = (e * Bt).sum(1)
            dec = e * a * hist[t]
            o["du"][t] = Dv * out + delta[t] * eB
            ddt = (eB * u[t] + (dec * A).sum(1)) * slope[t]
            o["ddt"][t] = ddt
            o["ddt_bias"] += ddt
            o["dA"] += dec * delta[t][:, None]
            o["dD"] += out * u[t]
            carry = e * a
        o["dS0"][b] = carry
    return o


# ---- group norm ----------------------------------------------------------------

def _normed(x, w, bias, G, eps, center):
    R, C = x.shape
    D = C // G
    xg = x.reshape(R, G, D)
    mu = xg.mean(2, keepdims=True) if center else np.zeros((R, G, 1))
    r = 1.0 / np.sqrt(((xg - mu) ** 2).mean(2, keepdims=True) + eps)
    full = lambda v, d: np.full((G, D), d) if v is None else np.broadcast_to(v.reshape(-1, D), (G, D))
    return xg, mu, r, full(w, 1.0), full(bias, 0.0)


def norm_forward(x, w, bias, z, G, eps, center, act, mag=False):
    """y"""
    xg, mu, r, wf, bf = _normed(x, w, bias, G, eps, center)
    xh = (xg - mu) * r
    n = xh * wf + bf
    zg = None if z is None else z.reshape(xg.shape)
    if mag:
        # xh: the subtraction loses 2^-24 (|x| + |mu|), the mean up to mean|x|
        xm = (np.abs(xg) + np.abs(xg).mean(2, keepdims=True)) * r if center else np.abs(xh)
        nm = xm * np.abs(wf) + np.abs(bf)
        if zg is None:
            return (1.1 * nm if act else nm).reshape(x.shape)
        return (nm * np.abs(silu(zg) if act else zg)).reshape(x.shape)
    if zg is None:
        y = silu(n) if act else n
    else:
        y = n * (silu(zg) if act else zg)
    return y.reshape(x.shape)


def norm_backward(x, w, bias, z, G, eps, center, act, dy, mag=False):
    """(dx, dw, dbias, dz); dw, dbias per channel [C]"""
    xg, mu, r, wf, bf = _normed(x, w, bias, G, eps, center)
    xh = (xg - mu) * r
    n = xh * wf + bf
    dyg = dy.reshape(xg.shape)
    zg = None if z is None else z.reshape(xg.shape)
    one = np.ones_like(xg)
    if zg is None:
        dn, dz = dyg * (dsilu(n) if act else one), None
    else:
        dn = dyg * (silu(zg) if act else zg)
        dz = dyg * n * (dsilu(zg) if act else one)
    if mag:
        xm = (np.abs(xg) + np.abs(xg).mean(2, keepdims=True)) * r if center else np.abs(xh)
        nm = xm * np.abs(wf) + np.abs(bf)
        if zg is None:
            # act' is off by at most 0.5 times the error of n
            dn = np.abs(dyg) * (np.abs(dsilu(n)) + 0.5 * nm if act else one)
        else:
            dn = np.abs(dn)
            dz = np.abs(dyg) * nm * (np.abs(dsilu(zg)) + 0.5 * np.abs(zg) if act else one)
        e = dn * np.abs(wf)
        dx = r * (e + (e.mean(2, keepdims=True) if center else 0.0) + xm * (e * xm).mean(2, keepdims=True))
        xh = xm
    else:
        e = dn * wf
        dx = r * (e - (e.mean(2, keepdims=True) if center else 0.0) - xh * (e * xh).mean(2, keepdims=True))
    shape = x.shape
    return (dx.reshape(shape), (dn * xh).sum(0).reshape(-1), dn.sum(0).reshape(-1),
            None if dz is None else dz.reshape(shape))
