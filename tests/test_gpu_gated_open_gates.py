"""Gradients of the gated recurrence where its gates are wide open or shut,
against 64 bits within bounds that shrink with what is left of a gate
(plain64_gates.py)."""
import numpy as np
import pytest

import plain64_gated as P
import plain64_gates as G
from test_gpu_gated_scan import _make
from test_gpu_linear_attn import _close, _np

pytestmark = pytest.mark.gpu


def _check(d, dy, dh, dtype, ckpt):
    import torch
    from selective_state_space_84_amd import binding as bd
    ck = bd.ssm_gated_scan_fwd(**d, want_ckpt=True)[2] if ckpt else None
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck)
    torch.cuda.synchronize()
    ref = G.gate_grads(**{k: _np(v) for k, v in d.items()}, dy=_np(dy), dh_last=_np(dh))
    for n in ("dga", "dgx"):
        _close(n, _np(g[n]), ref[n][0], P.tol(*ref[n], dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [8.0, 10.0, 12.0, 14.0, 17.0, 20.0, 30.0])
@pytest.mark.parametrize("z", [False, True])
def test_wide_open_gates(lib, z, gate, dtype):
    """One gate wide open, the other, or both, at every step of some channels; whole and partial pieces, one channel a
    lane and two."""
    r = np.random.default_rng(int(gate))
    for L, D in ((1, 96), (200, 96), (70, 33)):
        print("case", L, D, gate, z, dtype, flush=True)
        d, dy, dh = _make(L + D, 2, L, D, dtype, z=z)
        for name, every in (("ga", 2), ("gx", 3)):
            t = d[name][:, :, ::every]
            t.copy_(gate + t.new_tensor(r.uniform(-0.4, 0.4, tuple(t.shape))))
        _check(d, dy, dh, dtype, ckpt=L != 70)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_of_any_size(lib, dtype):
    """Gates from shut to open across a row, and beyond what e^-v holds in fp32 (where a gradient is below fp32's normal
    range and may be flushed)."""
    r = np.random.default_rng(0)
    d, dy, dh = _make(1, 2, 150, 64, dtype)
    for name in ("ga", "gx"):
        d[name].copy_(d[name].new_tensor(r.uniform(-40.0, 40.0, tuple(d[name].shape))))
    _check(d, dy, dh, dtype, ckpt=True)
    d["ga"][:, ::5], d["gx"][:, 1::5] = 100.0, 1000.0
    d["gx"][:, 2::5] = -100.0
    _check(d, dy, dh, dtype, ckpt=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
def test_sum_over_steps_ends_with_the_row(lib, z, dtype):
    """dlog_a sums a row's own steps, whatever reaches the steps behind them: with x = 0, h0 > 0 and an infinite
    gradient of the last state every step of a row adds +inf, and those behind it nothing (not inf * 0).  Where the
    decays of a row multiply to less than e^-80 (fp32 ends at e^-87), a state or a product of decays may be 0 in fp32
    and its product with inf NaN: such channels are left out."""
    import torch
    from selective_state_space_84_amd import binding as bd
    for n in (0, 1, 7, 8, 9, 63, 64, 65, 100, 128, 130):
        print("case", n, z, dtype, flush=True)
        d, dy, dh = _make(n, 1, 130, 70, dtype, z=z)
        d["x"].zero_()
        d["h0"].abs_().add_(1.0)
        dh.fill_(float("inf"))
        lens = torch.tensor([n], dtype=torch.int32, device=dy.device)
        g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, lengths=lens)
        la = (_np(d["log_a"]) * P.sigmoid(_np(d["ga"][0, :n]))).sum(0)
        kept = torch.as_tensor(la > -80.0, device=dy.device)
        assert kept.sum() >= 20 and (kept.all() or n > 9)
        assert (g["dlog_a"][kept] == (float("inf") if n else 0.0)).all(), n
        assert (g["dh0"][0, kept] == float("inf")).all(), n
