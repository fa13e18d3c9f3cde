"""The gated recurrence, the gated norm and the residual update with its norms,
and their gradients, in 64 bits on the CPU from the definitions, each with a
bound on the rounding errors of a computation in fp32.

Bounds.  U is half a step of fp32.  The hardware's exponential, reciprocal and
reciprocal root are off by one step (2 U), every product and sum by U:
  sigmoid(v): its exponential's argument is rounded (|v| U of the exponential,
     whose share in the result is 1 - sigmoid), then 2 + 1 + 2 roundings;
  log a = log_a sigmoid(ga): that and 3 more; a: |log a| times that, and 2;
  1 - a: a / (1 - a) |log a| <= 1, so log a's error again, and 9 at most;
  m = sqrt((1 - a)(1 + a)): that error again and 7 more.
A state's error follows the recurrence: what it had times a, the errors of a
(and 3 roundings a step, for products of decays that are formed apart) and of
the step's input, both relative to the same recurrence over absolute values.
Everything is then taken twice, for products of errors and other orders."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -126  # where 1 - a^2 is below, the input counts as nothing


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(v, dtype=np.float64)))


def silu(z):
    return z * sigmoid(z)


def sig_err(v):
    """Relative error of a sigmoid, in U."""
    return 6.0 + np.abs(v) * (1.0 - sigmoid(v))


def _count(lengths, L, b):
    return L if lengths is None else min(max(int(lengths[b]), 0), L)


def _parts(ga, gx, log_a):
    sa, sx = sigmoid(ga), sigmoid(gx)
    la = log_a * sa
    m2 = -np.expm1(2.0 * la)
    return sa, sx, la, np.exp(la), np.sqrt(np.where(m2 < TINY, 0.0, m2))


def scan(x, ga, gx, log_a, z=None, lengths=None, h0=None, dy=None, dh_last=None):
    """Outputs and, with dy, gradients of one call; a dict of (value, bound on the error before the last rounding)."""
    B, L, D = x.shape
    out = {"y": np.zeros((2, B, L, D)), "h_last": np.zeros((2, B, D))}
    grad = dy is not None
    if grad:
        for n in ("dx", "dga", "dgx", "dz"):
            out[n] = np.zeros((2, B, L, D))
        out["dh0"], out["dlog_a"] = np.zeros((2, B, D)), np.zeros((2, D))
        dlog_mag = np.zeros(D)
    for b in range(B):
        n = _count(lengths, L, b)
        s = slice(0, n)
        sa, sx, la, a, m = _parts(ga[b, s], gx[b, s], log_a)
        ra, rx = sig_err(ga[b, s]), sig_err(gx[b, s])
        al = np.abs(la) * (ra + 3) + 2
        w = sx * x[b, s]
        u, ru = m * w, ra + rx + 20
        h, H, E = (np.zeros((n + 1, D)) for _ in range(3))
        if h0 is not None:
            h[0], H[0] = h0[b], np.abs(h0[b])
        for t in range(n):
            h[t + 1] = a[t] * h[t] + u[t]
            H[t + 1] = a[t] * H[t] + np.abs(u[t])
            E[t + 1] = a[t] * E[t] + U * ((al[t] + 3) * a[t] * H[t] + ru[t] * np.abs(u[t]))
        out["h_last"][:, b] = h[n], E[n]
        if z is None:
            gate, rz = np.ones((n, D)), np.zeros((n, D))
        else:
            gate, rz = silu(z[b, s]), sig_err(z[b, s]) + 1
        out["y"][0, b, s] = h[1:] * gate
        out["y"][1, b, s] = np.abs(gate) * (E[1:] + U * (rz + 1) * H[1:])
        if not grad:
            continue
        e = dy[b, s] * gate
        g, G, F = (np.zeros((n + 1, D)) for _ in range(3))  # of the state behind each step; last: behind the row
        p = np.zeros((3, D))  # what reaches it from the step behind, its magnitude and error
        if dh_last is not None:
            p[0], p[1] = dh_last[b], np.abs(dh_last[b])
        for t in reversed(range(n)):
            g[t], G[t] = e[t] + p[0], np.abs(e[t]) + p[1]
            F[t] = U * (rz[t] + 2) * np.abs(e[t]) + p[2]
            p = np.stack([a[t] * g[t], a[t] * G[t], a[t] * (F[t] + U * (al[t] + 3) * G[t])])
        g, G, F = g[:n], G[:n], F[:n]
        out["dh0"][:, b] = p[0], p[2]
        gm, GM = g * m, G * m
        FM = m * F + U * (ra + 17) * GM
        fx = sx * (FM + U * (rx + 1) * GM)
        out["dx"][0, b, s], out["dx"][1, b, s] = gm * sx, fx
        xx = np.abs(x[b, s])
        out["dgx"][0, b, s] = gm * sx * x[b, s] * (1 - sx)
        out["dgx"][1, b, s] = xx * ((1 - sx) * fx + GM * sx * U * (sx * rx + 1 + 2 * (1 - sx)))
        with np.errstate(divide="ignore", invalid="ignore"):
            k = np.where(m > 0, a * a / m, 0.0)
        dla = g * (a * h[:-1] - k * w)
        q1, q2 = a * H[:-1], k * np.abs(w)
        fla = F * (q1 + q2) + G * (a * E[:-1] + U * (q1 * (al + 4) + q2 * (2 * al + ra + rx + 26)))
        mla = G * (q1 + q2)
        out["dga"][0, b, s] = dla * log_a * sa * (1 - sa)
        out["dga"][1, b, s] = np.abs(log_a) * sa * ((1 - sa) * fla + mla * U * (sa * ra + 1 + (ra + 4) * (1 - sa)))
        out["dlog_a"][0] += (dla * sa).sum(0)
        out["dlog_a"][1] += (sa * (fla + U * (ra + 1) * mla)).sum(0)
        dlog_mag += (sa * mla).sum(0)
        if z is not None:
            zz, sz = z[b, s], sigmoid(z[b, s])
            slope = sz * (1 + zz * (1 - sz))
            out["dz"][0, b, s] = dy[b, s] * h[1:] * slope
            out["dz"][1, b, s] = np.abs(dy[b, s]) * (E[1:] * np.abs(slope) + H[1:] * U * (
                np.abs(slope) * (rz + 3) + sz * (np.abs(zz) * (sz * rz + 2) + 1)))
    if grad:
        out["dlog_a"][1] += U * (B * L + 16) * dlog_mag
    return out


def tol(ref, bound, dtype):
    """Bound on a stored output's error; 1e-30: values below fp32's normal range may be flushed."""
    return HALF[dtype] * np.abs(ref) + 2.0 * bound + 1e-30


def update(h, x, ga, gx, log_a, z=None, slots=None):
    """One step on h (n_slots, D): (y, h) with their bounds."""
    B, D = x.shape
    y, hn = np.zeros((2, B, D)), np.stack([np.array(h, dtype=np.float64), np.zeros(h.shape)])
    for b in range(B):
        k = b if slots is None else int(slots[b])
        if not 0 <= k < h.shape[0]:
            continue
        r = scan(x[b][None, None], ga[b][None, None], gx[b][None, None], log_a,
                 None if z is None else z[b][None, None], h0=h[k][None])
        y[:, b], hn[:, k] = r["y"][:, 0, 0], r["h_last"][:, 0]
    return y, hn


# ---- norms -----------------------------------------------------------------

def _root(t, eps):
    return 1.0 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)


def gated_norm(x, z, w, groups, gate_first, eps, dy=None):
    """x, z, dy: (rows, width).  A dict of (value, bound): y, and with dy dx, dz, dw."""
    rows, width = x.shape
    G = width // groups
    split = lambda v: v.reshape(rows, groups, G)  # noqa: E731
    w = np.ones(width) if w is None else w
    gate, sz = (np.ones_like(x), np.ones_like(x)) if z is None else (silu(z), sigmoid(z))
    rz = np.zeros_like(x) if z is None else sig_err(z) + 1
    t = split(x * gate if gate_first else x)
    r = _root(t, eps)
    n = (t * r).reshape(rows, width) * w
    y = n if gate_first else n * gate
    top = split(rz).max(-1, keepdims=True).repeat(G, -1).reshape(rows, width)
    out = {"y": (y, U * (G + 3 * top + 16) * np.abs(y))}
    if dy is None:
        return out
    g = split((dy if gate_first else dy * gate) * w)
    c = (g * t).mean(-1, keepdims=True) * r * r
    C = np.abs(g * t).mean(-1, keepdims=True) * r * r
    dt = (r * (g - t * c)).reshape(rows, width)
    dtm = (r * (np.abs(g) + np.abs(t) * C)).reshape(rows, width)
    k = U * (3 * G + 6 * top + 32)
    if z is None:
        out["dx"] = (dt, k * dtm)
    else:
        slope, slope_mag = sz * (1 + z * (1 - sz)), sz * (1 + np.abs(z))
        more = U * (2 * rz + 6)
        if gate_first:
            out["dx"] = (dt * gate, (k + more) * dtm * np.abs(gate))
            out["dz"] = (dt * x * slope, np.abs(x) * dtm * (k * np.abs(slope) + more * slope_mag))
        else:
            out["dx"] = (dt, k * dtm)
            out["dz"] = (dy * n * slope, np.abs(dy * n) * (k * np.abs(slope) + more * slope_mag))
    terms = (dy if gate_first else dy * gate) * (t * r).reshape(rows, width)
    out["dw"] = (terms.sum(0), U * ((rows + G + 16) * np.abs(terms) + 6 * top * np.abs(terms)).sum(0))
    return out


def residual_norm(x, res, w_pre, w_post, alpha, post_norm, eps):
    """A dict of (value, bound): res_out, y."""
    D = x.shape[-1]
    w_pre, w_post = (np.ones(D) if w is None else w for w in (w_pre, w_post))
    n = w_post * (x * _root(x, eps) if post_norm else x)
    res = np.zeros_like(x) if res is None else res
    R = res + alpha * n
    mag = np.abs(res) + np.abs(alpha * n)
    e = U * (D + 16) * np.abs(alpha * n) + 2 * U * mag
    r = _root(R, eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        share = (np.abs(R) * e).sum(-1, keepdims=True) / ((R * R).sum(-1, keepdims=True) + D * eps)
    y = R * r * w_pre
    return {"res_out": (R, e), "y": (y, r * np.abs(w_pre) * e + np.abs(y) * (share + U * (D + 16)))}


def residual_norm_bwd(x, R, w_pre, w_post, dy, dres_out, alpha, post_norm, eps):
    """A dict of (value, bound): dx, dres, dw_pre, dw_post."""
    rows, D = R.shape
    w_pre, w_post = (np.ones(D) if w is None else w for w in (w_pre, w_post))
    dres_out = np.zeros_like(R) if dres_out is None else dres_out
    r = _root(R, eps)
    g = dy * w_pre
    G = r * (g - R * (g * R).mean(-1, keepdims=True) * r * r) + dres_out
    M = r * (np.abs(g) + np.abs(R) * np.abs(g * R).mean(-1, keepdims=True) * r * r) + np.abs(dres_out)
    e = U * (3 * D + 32) * M
    out = {"dres": (G, e)}
    t1 = dy * R * r
    out["dw_pre"] = (t1.sum(0), U * (rows + D + 16) * np.abs(t1).sum(0))
    g2, m2 = alpha * G * w_post, np.abs(alpha * w_post) * M
    if not post_norm:
        out["dx"] = (g2, np.abs(alpha * w_post) * e + 2 * U * m2)
        if x is not None:
            t2, a2 = alpha * G * x, np.abs(alpha * x) * M
            out["dw_post"] = (t2.sum(0), (U * (rows + 3 * D + 48) * a2).sum(0))
        return out
    q = _root(x, eps)
    out["dx"] = (q * (g2 - x * (g2 * x).mean(-1, keepdims=True) * q * q),
                 U * (6 * D + 64) * q * (m2 + np.abs(x) * (m2 * np.abs(x)).mean(-1, keepdims=True) * q * q))
    t2, a2 = alpha * G * x * q, np.abs(alpha * x) * M * q
    out["dw_post"] = (t2.sum(0), (U * (rows + 4 * D + 64) * a2).sum(0))
    return out
