"""Linear attention, the query/key norm with rotation, and their gradients in
64 bits on the CPU, one step and one head at a time from the definitions, with
the magnitude every output's rounding errors scale with.

Magnitudes: the same sums over absolute values, each decayed term counted
1 + x times for a decay of 2^-x (an exponent of x is formed with a relative
error, so its power's error grows with x)."""
import math

import numpy as np

U = 2.0 ** -24      # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _weights(g, d):
    """exp(g d) for d >= 0 (1 at d = 0 whatever g), 0 for d < 0; and the same times 1 + x."""
    dd = np.maximum(d, 0).astype(np.float64)
    with np.errstate(invalid="ignore"):
        e = np.where(dd == 0, 0.0, g * dd)
    w = np.where(d >= 0, np.exp(e), 0.0)
    x = np.where(np.isfinite(e), np.abs(e) / math.log(2.0), 0.0)
    return w, w * (1.0 + x)


def attn_fwd(q, k, v, log_decay, lengths=None, h0=None, scale=None):
    """Step by step; returns (o, h_last)."""
    B, L, H, K = q.shape
    M, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    o = np.zeros((B, L, H, V))
    hl = np.zeros((B, H, V, K)) if h0 is None else np.array(h0, dtype=np.float64)
    gam = np.exp(np.asarray(log_decay, dtype=np.float64))
    for b in range(B):
        for h in range(H):
            m = h // (H // M)
            for t in range(L if lengths is None else min(max(int(lengths[b]), 0), L)):
                hl[b, h] = gam[h] * hl[b, h] + np.outer(v[b, t, m], k[b, t, m])
                o[b, t, h] = scale * (hl[b, h] @ q[b, t, h])
    return o, hl


def attn_bwd(q, k, v, log_decay, do, lengths=None, h0=None, dh_last=None, scale=None):
    """Reverse mode, step by step; returns (dq, dk, dv, dh0)."""
    B, L, H, K = q.shape
    M, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dh0 = np.zeros((B, H, V, K))
    gam = np.exp(np.asarray(log_decay, dtype=np.float64))
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for h in range(H):
            m = h // (H // M)
            st = np.zeros((V, K)) if h0 is None else np.array(h0[b, h], dtype=np.float64)
            for t in range(n):
                st = gam[h] * st + np.outer(v[b, t, m], k[b, t, m])
                dq[b, t, h] = scale * (st.T @ do[b, t, h])
            G = np.zeros((V, K)) if dh_last is None else np.array(dh_last[b, h], dtype=np.float64)
            for t in reversed(range(n)):
                G = G + scale * np.outer(do[b, t, h], q[b, t, h])
                dk[b, t, m] += G.T @ v[b, t, m]
                dv[b, t, m] += G @ k[b, t, m]
                G = gam[h] * G
            dh0[b, h] = G
    return dq, dk, dv, dh0


def _mag(a, b, c, g, n, entry, s_pair, s_read, s_write, rev):
    """Magnitudes of sum_i w |a_t|.|b_i| |c_i| + entry's share, and of the state left; one head, n steps."""
    a, b, c = np.abs(a[:n]), np.abs(b[:n]), np.abs(c[:n])
    t = np.arange(n)
    d = t[:, None] - t[None, :]
    w = _weights(g, -d if rev else d)[1]
    out = s_pair * ((a @ b.T) * w) @ c
    r = _weights(g, (n - 1 - t) if rev else t + 1)[1]
    out = out + s_read * r[:, None] * (a @ np.abs(entry))
    u = _weights(g, t + 1 if rev else n - 1 - t)[1]
    st = _weights(g, np.array(n))[1] * np.abs(entry) + s_write * (b * u[:, None]).T @ c
    return out, st


def attn_fwd_mag(q, k, v, log_decay, lengths=None, h0=None, scale=None):
    B, L, H, K = q.shape
    M, V = v.shape[2:]
    scale = abs(K ** -0.5 if scale is None else scale)
    o, hl = np.zeros((B, L, H, V)), np.zeros((B, H, V, K))
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for h in range(H):
            m = h // (H // M)
            e = np.zeros((K, V)) if h0 is None else h0[b, h].T
            o[b, :n, h], st = _mag(q[b, :, h], k[b, :, m], v[b, :, m], log_decay[h], n, e, scale, scale, 1.0, False)
            hl[b, h] = st.T
    return o, hl


def attn_bwd_mag(q, k, v, log_decay, do, lengths=None, h0=None, dh_last=None, scale=None):
    B, L, H, K = q.shape
    M, V = v.shape[2:]
    sc = abs(K ** -0.5 if scale is None else scale)
    dq, dk, dv, dh0 = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros((B, H, V, K))
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for h in range(H):
            m = h // (H // M)
            e = np.zeros((V, K)) if h0 is None else h0[b, h]
            f = np.zeros((V, K)) if dh_last is None else dh_last[b, h]
            g = log_decay[h]
            dq[b, :n, h] = _mag(do[b, :, h], v[b, :, m], k[b, :, m], g, n, e, sc, sc, 1.0, False)[0]
            dk[b, :n, m] += _mag(v[b, :, m], do[b, :, h], q[b, :, h], g, n, f, sc, 1.0, sc, True)[0]
            out, st = _mag(k[b, :, m], q[b, :, h], do[b, :, h], g, n, f.T, sc, 1.0, sc, True)
            dv[b, :n, m] += out
            dh0[b, h] = st.T
    return dq, dk, dv, dh0


def attn_tol(out, mag, steps, width, dtype, rep=1):
    """Bound on an output's error.  fp32: every product and sum of its steps x
    width terms rounds once (taken twice as coarse, for sums inside the matrix
    instructions), the decays' powers count in mag.  bf16 outputs round once at
    the end, and operands carried as two bf16 values are off by 2^-16."""
    fp32 = (steps + width + rep + 16) * 2 * U * mag
    if dtype == "f32":
        return HALF["f32"] * np.abs(out) + fp32
    return HALF["bf16"] * np.abs(out) + 2 * 2.0 ** -16 * mag + fp32


# ---- norm and rotation ---------------------------------------------------

def _angles(pos, inv_freq):
    a = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    return np.cos(a), np.sin(a)


def _pairs(R, interleaved):
    j = np.arange(R // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)


def rotate(x, pos, inv_freq, interleaved, back=False):
    """x (B, L, H, D) at positions (B, L)."""
    R = 2 * len(inv_freq)
    out = np.array(x, dtype=np.float64)
    if R == 0:
        return out
    cos, sin = (c[:, :, None, :] for c in _angles(pos, inv_freq))
    if back:
        sin = -sin
    i, j = _pairs(R, interleaved)
    out[..., i] = x[..., i] * cos - x[..., j] * sin
    out[..., j] = x[..., i] * sin + x[..., j] * cos
    return out


def rotate_mag(x, R, interleaved):
    out = np.abs(x)
    if R:
        i, j = _pairs(R, interleaved)
        s = np.abs(x[..., i]) + np.abs(x[..., j])
        out[..., i] = s
        out[..., j] = s
    return out


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """(values, magnitudes)"""
    D = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r * (np.ones(D) if w is None else w)
    return rotate(n, pos, inv_freq, interleaved), rotate_mag(n, 2 * len(inv_freq), interleaved)


def norm_rope_bwd(x, w, pos, inv_freq, eps, interleaved, dy):
    """(dx, dw, magnitude of dx, magnitude of dw)"""
    D = x.shape[-1]
    w = np.ones(D) if w is None else w
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = rotate(dy, pos, inv_freq, interleaved, back=True)
    gm = rotate_mag(dy, 2 * len(inv_freq), interleaved)
    dx = r * w * g - x * r ** 3 * (w * g * x).mean(-1, keepdims=True)
    dxm = r * np.abs(w) * gm + np.abs(x) * r ** 3 * (np.abs(w * x) * gm).mean(-1, keepdims=True)
    ax = (0, 1, 2)
    return dx, (g * x * r).sum(ax), dxm, (gm * np.abs(x) * r).sum(ax)
