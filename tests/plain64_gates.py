"""Gradients of the gated recurrence's two gates in 64 bits, with bounds on the
rounding errors that stay relative where a gate is wide open.

A gate's gradient has the factor s (1 - s), s its sigmoid.  1 - s is
sigmoid(-v) = e / (1 + e) with e = e^-v, here and in fp32: a product and a
reciprocal, none of which cancels, so its relative error in U is that of a
sigmoid at -v (plain64_gated.sig_err).  The bounds of the other factors are those of
plain64_gated.py: of the gradient of the input (dgx), and of the gradient of
log a (dga).  Products of the kernel: u (1 - s), g times that and u itself for
dgx; log_a (1 - s), its product, and five in what it multiplies for dga."""
import numpy as np

import plain64_gated as P


def gate_grads(x, ga, gx, log_a, dy, z=None, h0=None, dh_last=None):
    """{dga, dgx: (value, bound on the error before the last rounding)}; every row whole."""
    B, L, D = x.shape
    out = {n: np.zeros((2, B, L, D)) for n in ("dga", "dgx")}
    for b in range(B):
        sa, sx, la, a, m = P._parts(ga[b], gx[b], log_a)
        shut_a, shut_x = P.sigmoid(-ga[b]), P.sigmoid(-gx[b])
        ra, rx = P.sig_err(ga[b]), P.sig_err(gx[b])
        al = np.abs(la) * (ra + 3) + 2
        w = sx * x[b]
        u, ru = m * w, ra + rx + 20
        h, H, E = (np.zeros((L + 1, D)) for _ in range(3))
        if h0 is not None:
            h[0], H[0] = h0[b], np.abs(h0[b])
        for t in range(L):
            h[t + 1] = a[t] * h[t] + u[t]
            H[t + 1] = a[t] * H[t] + np.abs(u[t])
            E[t + 1] = a[t] * E[t] + P.U * ((al[t] + 3) * a[t] * H[t] + ru[t] * np.abs(u[t]))
        e, rz = dy[b], np.zeros((L, D))
        if z is not None:
            e, rz = dy[b] * P.silu(z[b]), P.sig_err(z[b]) + 1
        g, G, F = (np.zeros((L, D)) for _ in range(3))
        p = np.zeros((3, D))
        if dh_last is not None:
            p[0], p[1] = dh_last[b], np.abs(dh_last[b])
        for t in reversed(range(L)):
            g[t], G[t] = e[t] + p[0], np.abs(e[t]) + p[1]
            F[t] = P.U * (rz[t] + 2) * np.abs(e[t]) + p[2]
            p = np.stack([a[t] * g[t], a[t] * G[t], a[t] * (F[t] + P.U * (al[t] + 3) * G[t])])
        gm, GM = g * m, G * m
        fx = sx * (m * F + P.U * (ra + 17) * GM + P.U * (rx + 1) * GM)
        out["dgx"][0, b] = gm * w * shut_x
        out["dgx"][1, b] = np.abs(x[b]) * shut_x * (fx + GM * sx * P.U * (P.sig_err(-gx[b]) + 3))
        with np.errstate(divide="ignore", invalid="ignore"):
            k = np.where(m > 0, a * a / m, 0.0)
        q1, q2 = a * H[:-1], k * np.abs(w)
        fla = F * (q1 + q2) + G * (a * E[:-1] + P.U * (q1 * (al + 4) + q2 * (2 * al + ra + rx + 26)))
        mla = G * (q1 + q2)
        out["dga"][0, b] = g * (a * h[:-1] - k * w) * log_a * sa * shut_a
        out["dga"][1, b] = np.abs(log_a) * sa * shut_a * (fla + mla * P.U * (ra + P.sig_err(-ga[b]) + 8))
    return out
