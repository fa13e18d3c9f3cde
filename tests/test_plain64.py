"""The 64-bit definitions of linear attention and of the norm with rotation
(plain64.py) against differences and closed forms, on the CPU."""
import numpy as np
import pytest

import plain64 as P


def _attn(seed, B=2, L=6, H=4, M=2, K=3, V=5):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(q=n((B, L, H, K)), k=n((B, L, M, K)), v=n((B, L, M, V)), log_decay=-np.abs(n(H)) * 0.5,
                h0=n((B, H, V, K))), n((B, L, H, V)), n((B, H, V, K))


@pytest.mark.parametrize("lengths", [None, [6, 3], [0, 1]])
def test_attn_gradient_against_differences(lengths):
    a, do, dh = _attn(1)

    def loss():
        o, hl = P.attn_fwd(lengths=lengths, **a)
        return (o * do).sum() + (hl * dh).sum()
    grads = dict(zip(("q", "k", "v", "h0"), P.attn_bwd(do=do, dh_last=dh, lengths=lengths, **a)))
    for name, g in grads.items():
        x = a[name]
        num = np.zeros(x.shape)
        for i in np.ndindex(x.shape):
            old = x[i]
            x[i] = old + 1e-4
            up = loss()
            x[i] = old - 1e-4
            num[i] = (up - loss()) / 2e-4
            x[i] = old
        # The loss is linear in each single element: differences only round.
        assert np.abs(num - g).max() <= 1e-8 * max(1.0, np.abs(g).max()), name


def test_attn_is_decayed_pairs():
    a, _, _ = _attn(2)
    o, _ = P.attn_fwd(**a)
    B, L, H, K = a["q"].shape
    for h in range(H):
        g = a["log_decay"][h]
        d = np.arange(L)[:, None] - np.arange(L)[None, :]
        w = np.where(d >= 0, np.exp(g * np.maximum(d, 0)), 0)
        for b in range(B):
            q, k, v = a["q"][b, :, h], a["k"][b, :, h // 2], a["v"][b, :, h // 2]
            want = ((q @ k.T) * w) @ v + np.exp(g * (np.arange(L) + 1))[:, None] * (q @ a["h0"][b, h].T)
            assert np.allclose(o[b, :, h], want * K ** -0.5, rtol=1e-12, atol=1e-12)


def test_attn_decay_limits():
    a, _, _ = _attn(3)
    a["log_decay"] = np.full(4, -np.inf)  # only the current step
    o, hl = P.attn_fwd(**a)
    for h in range(4):
        m = h // 2
        want = (a["q"][:, :, h] * a["k"][:, :, m]).sum(-1)[..., None] * a["v"][:, :, m] * 3 ** -0.5
        assert np.allclose(o[:, :, h], want)
    m = P.attn_fwd_mag(**a)
    assert np.isfinite(m[0]).all() and np.isfinite(m[1]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_gradient_against_differences(interleaved, rot):
    r = np.random.default_rng(4)
    x, w, dy = r.standard_normal((2, 3, 2, 8)), r.standard_normal(8), r.standard_normal((2, 3, 2, 8))
    pos, f = r.integers(0, 50, (2, 3)), r.random(rot // 2)

    def loss():
        return (P.norm_rope(x, w, pos, f, 1e-3, interleaved)[0] * dy).sum()
    dx, dw, _, _ = P.norm_rope_bwd(x, w, pos, f, 1e-3, interleaved, dy)
    for arr, g in ((x, dx), (w, dw)):
        num = np.zeros(arr.shape)
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + 1e-5
            up = loss()
            arr[i] = old - 1e-5
            num[i] = (up - loss()) / 2e-5
            arr[i] = old
        # Central differences: 1e-10 times third derivatives of order 10, and rounding of 1e-16 / 1e-5.
        assert np.abs(num - g).max() <= 1e-7


def test_rotation_keeps_length_and_relative_positions():
    r = np.random.default_rng(5)
    a, b, f = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8)), r.random(4)
    at = lambda x, p: P.rotate(x, [[p]], f, False)
    assert np.allclose((at(a, 9) ** 2).sum(), (a ** 2).sum())
    assert np.allclose((at(a, 9) * at(b, 4)).sum(), (at(a, 105) * at(b, 100)).sum())
    assert np.allclose(P.rotate(at(a, 7), [[7]], f, False, back=True), a)
