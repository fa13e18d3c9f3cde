"""Gated norm and residual norm at both ends of the values that they take,
with groups of every plan up to the widest: |t| up to 10^18, and with eps 0 a
root mean square down to 10^-18, against the 64-bit definitions within the
bounds of plain64_gated.py."""
import numpy as np
import pytest

import plain64_gated as P
from test_gpu_linear_attn import _close, _np, _t

pytestmark = pytest.mark.gpu

GROUPS = [(8, 1), (100, 1), (512, 1), (1024, 2), (1001, 1), (4096, 1), (8192, 1), (16384, 1), (16383, 1)]
# Sizes of the values: all but at the upper end in every place, and a little above the lower end.
ENDS = [(9.9e17, 1e-6), (9.9e17, 0.0), (1.3e-18, 0.0)]


def _values(r, rows, D, size):
    """Of one size and either sign."""
    return size * np.where(r.random((rows, D)) < 0.5, -1.0, 1.0)


def _held(got, ref, types):
    for n, v in got.items():
        want, e = (a.reshape(v.shape) for a in ref[n])
        assert np.isfinite(want).all()
        _close(n, _np(v), want, P.tol(want, e, types[n]))
        assert np.abs(_np(v)).max() > 0, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", ENDS)
def test_gated_norm(lib, size, eps, dtype):
    import torch
    from selective_state_space_84_amd import binding as bd
    for D, groups in GROUPS:
        for gate, first in ((False, True), (True, True), (True, False)):
            print("case", D, groups, size, eps, gate, first, dtype, flush=True)
            r = np.random.default_rng(D)
            # A gate of 1.2784645 has silu 1 (0.99... in bf16): t keeps its size.
            x, z = _t(_values(r, 5, D, size), dtype), (_t(np.full((5, D), 1.2784645), dtype) if gate else None)
            w, dy = _t(1 + 0.3 * r.standard_normal(D)), _t(r.standard_normal((5, D)), dtype)
            y = bd.ssm_gated_norm_fwd(x, z, w, groups=groups, gate_first=first, eps=eps)
            g = bd.ssm_gated_norm_bwd(x, z, w, dy=dy, groups=groups, gate_first=first, eps=eps)
            torch.cuda.synchronize()
            _held({"y": y, **g}, P.gated_norm(_np(x), _np(z), _np(w), groups, first, eps, _np(dy)),
                  {"y": dtype, "dx": dtype, "dz": dtype, "dw": "f32"})


@pytest.mark.parametrize("dtype,rt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("size,eps", ENDS)
def test_residual_norm(lib, size, eps, dtype, rt):
    import torch
    from selective_state_space_84_amd import binding as bd
    for D, _ in GROUPS:
        for post in (False, True):
            print("case", D, size, eps, post, dtype, rt, flush=True)
            r = np.random.default_rng(D)
            # Both norms' values are of the size: the stream is, and what is added takes an eighth of it away (alpha
            # brings the normed x there).
            al = -float(np.float32(0.125 * size if post else 0.125))
            x = _t(_values(r, 5, D, size), dtype)
            res = _t(size * np.sign(_np(x)), rt)
            wp, wo = _t(1 + 0.1 * r.uniform(-1, 1, D)), _t(1 + 0.1 * r.uniform(-1, 1, D))
            dy = _t(r.standard_normal((5, D)), dtype)
            R, y = bd.ssm_residual_norm_fwd(x, res, wp, wo, alpha=al, post_norm=post, eps=eps)
            g = bd.ssm_residual_norm_bwd(x, R, wp, wo, dy=dy, alpha=al, post_norm=post, eps=eps)
            torch.cuda.synchronize()
            _held({"res_out": R, "y": y}, P.residual_norm(_np(x), _np(res), _np(wp), _np(wo), al, post, eps),
                  {"res_out": rt, "y": dtype})
            _held(g, P.residual_norm_bwd(_np(x), _np(R), _np(wp), _np(wo), _np(dy), None, al, post, eps),
                  {"dx": dtype, "dres": rt, "dw_pre": "f32", "dw_post": "f32"})
