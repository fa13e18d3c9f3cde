"""Pins of the 64-bit definitions: closed forms, and every gradient against
central differences of the outputs (CPU)."""
import numpy as np
import pytest

import plain64_gated as P


def _ins(seed, B=2, L=5, D=3, z=True):
    r = np.random.default_rng(seed)
    d = dict(x=r.standard_normal((B, L, D)), ga=r.standard_normal((B, L, D)), gx=r.standard_normal((B, L, D)),
             log_a=-np.exp(r.uniform(-3, 1, D)), h0=r.standard_normal((B, D)))
    if z:
        d["z"] = r.standard_normal((B, L, D))
    return d, r


def _against_differences(loss, ins, grads):
    """Every element; central differences of step 1e-5 are off by h^2 f''' / 6 + eps f / h, 1e-9 of the loss's terms."""
    for name, g in grads.items():
        v = ins[name]
        for i in np.ndindex(v.shape):
            old = v[i]
            v[i] = old + 1e-5
            up = loss()
            v[i] = old - 1e-5
            down = loss()
            v[i] = old
            assert abs((up - down) / 2e-5 - g[i]) < 1e-6 * (1 + abs(g[i])), (name, i)


@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 3], [0, 4]])
def test_scan_gradient_against_differences(z, lengths):
    d, r = _ins(1, z=z)
    dy, dh = r.standard_normal((2, 5, 3)), r.standard_normal((2, 3))
    out = P.scan(**d, lengths=lengths, dy=dy, dh_last=dh)

    def loss():
        o = P.scan(**d, lengths=lengths)
        return (o["y"][0] * dy).sum() + (o["h_last"][0] * dh).sum()
    _against_differences(loss, d, {n: out["d" + n][0] for n in d})
    for b, n in enumerate(lengths or []):
        assert not out["y"][0][b, n:].any() and not out["dx"][0][b, n:].any() and not out["dga"][0][b, n:].any()


def test_scan_closed_forms():
    """Open gates and constant input: h_t = m x (1 - a^t) / (1 - a); shut gates keep the state."""
    D, L = 4, 50
    big = np.full((1, L, D), 60.0)
    log_a = -np.array([0.01, 0.3, 1.0, 4.0])
    a = np.exp(log_a)
    o = P.scan(np.ones((1, L, D)), big, big, log_a)
    t = np.arange(1, L + 1)[:, None]
    assert np.allclose(o["y"][0][0], np.sqrt(1 - a * a) * (1 - a ** t) / (1 - a), rtol=1e-12)
    h0 = np.arange(1.0, 5.0)[None]
    o = P.scan(np.ones((1, L, D)), -800 + big, big, log_a, h0=h0)
    assert np.allclose(o["h_last"][0], h0, rtol=1e-12)


def test_update_is_a_scan_of_one_step():
    d, r = _ins(2, B=3, L=1)
    h = r.standard_normal((5, 3))
    y, hn = P.update(h, d["x"][:, 0], d["ga"][:, 0], d["gx"][:, 0], d["log_a"], d["z"][:, 0], [4, -1, 1])
    o = P.scan(**{**d, "h0": np.stack([h[4], h[0], h[1]])})
    assert np.array_equal(y[0][[0, 2]], o["y"][0][[0, 2], 0]) and not y[0][1].any()
    assert np.array_equal(hn[0][[4, 1]], o["h_last"][0][[0, 2]]) and np.array_equal(hn[0][[0, 2, 3]], h[[0, 2, 3]])


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_norm_gradient_against_differences(groups, z, first):
    r = np.random.default_rng(3)
    d = dict(x=r.standard_normal((3, 6)), z=r.standard_normal((3, 6)) if z else None, w=r.standard_normal(6))
    dy = r.standard_normal((3, 6))
    out = P.gated_norm(**d, groups=groups, gate_first=first, eps=1e-2, dy=dy)
    _against_differences(lambda: (P.gated_norm(**d, groups=groups, gate_first=first, eps=1e-2)["y"][0] * dy).sum(), d,
                         {n: out["d" + n][0] for n in d if d[n] is not None})


@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_gradient_against_differences(post):
    r = np.random.default_rng(4)
    d = dict(x=r.standard_normal((3, 6)), res=r.standard_normal((3, 6)), w_pre=r.standard_normal(6),
             w_post=r.standard_normal(6))
    dy, dR = r.standard_normal((3, 6)), r.standard_normal((3, 6))
    k = dict(alpha=0.6, post_norm=post, eps=1e-2)
    o = P.residual_norm(**d, **k)
    g = P.residual_norm_bwd(d["x"], o["res_out"][0], d["w_pre"], d["w_post"], dy, dR, **k)

    def loss():
        q = P.residual_norm(**d, **k)
        return (q["y"][0] * dy).sum() + (q["res_out"][0] * dR).sum()
    _against_differences(loss, d, {"x": g["dx"][0], "res": g["dres"][0], "w_pre": g["dw_pre"][0],
                                   "w_post": g["dw_post"][0]})


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    assert np.allclose(P.gated_norm(x, None, None, 1, True, 0.0)["y"][0], [[1.2, 1.6, 0, 0]])
    want = [[3 / np.sqrt(13.5), 4 / np.sqrt(13.5), 0, 0]]
    assert np.allclose(P.gated_norm(x, None, None, 2, True, 1.0)["y"][0], want)
    o = P.residual_norm(x, np.array([[1.0, 1.0, 1.0, 1.0]]), None, np.array([1.0, 2.0, 1.0, 1.0]), 0.5, True, 0.0)
    assert np.allclose(o["res_out"][0], [[1.6, 2.6, 1.0, 1.0]])
