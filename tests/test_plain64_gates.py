"""The 64-bit gradients of plain64_gates.py: against the ones of plain64_gated.py where gates are half open, and
against closed forms where they are wide open."""
import numpy as np
import pytest

import plain64_gated as P
import plain64_gates as G


def _make(seed, B, L, D, gate):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    return dict(x=n(B, L, D), ga=gate(r, (B, L, D)), gx=gate(r, (B, L, D)), log_a=-np.exp(r.uniform(-4, 1, D)),
                z=n(B, L, D), h0=n(B, D), dy=n(B, L, D), dh_last=n(B, D))


@pytest.mark.parametrize("L", [1, 2, 30])
def test_half_open_gates(L):
    d = _make(L, 2, L, 6, lambda r, s: 2 * r.standard_normal(s))
    ref, got = P.scan(**d), G.gate_grads(**d)
    for n in ("dga", "dgx"):
        assert np.allclose(got[n][0], ref[n][0], rtol=1e-12, atol=1e-13), n


@pytest.mark.parametrize("gate", [8.0, 15.0, 30.0])
def test_wide_open_gates(gate):
    """One step: h = a h0 + m s x and L = h, whose derivatives are e^-gate of a simple product, and a little."""
    x, h0, log_a = 1.5, -0.7, -0.3
    one = np.ones((1, 1, 1))
    for which in ("ga", "gx"):
        v = dict(ga=0.4 * one, gx=-0.2 * one)
        v[which] = gate * one
        got = G.gate_grads(x=x * one, log_a=log_a * np.ones(1), dy=one, h0=h0 * np.ones((1, 1)), **v)[
            "d" + which][0].item()
        sa, sx = P.sigmoid(v["ga"]).item(), P.sigmoid(v["gx"]).item()
        a = np.exp(log_a * sa)
        m = np.sqrt(1 - a * a)
        s = sx if which == "gx" else sa
        slope = np.exp(-gate) * s * s  # s (1 - s)
        want = m * x * slope if which == "gx" else (a * h0 - a * a / m * sx * x) * log_a * slope
        assert abs(got - want) <= 1e-11 * abs(want)


def test_bounds_are_relative_to_what_is_left_of_a_gate():
    """A step further into saturation shrinks the bound as it shrinks the gradient."""
    for gate in (10.0, 20.0, 30.0):
        d = _make(3, 1, 20, 8, lambda r, s: gate + 0.1 * r.standard_normal(s))
        d["dy"], d["dh_last"] = np.abs(d["dy"]), np.abs(d["dh_last"])
        d["z"] = None
        v, e = G.gate_grads(**d)["dgx"]
        assert (e <= 200 * P.U * np.maximum(np.abs(v), 1e-300)).mean() > 0.9
