"""Gated norm and residual norm, and their gradients, against the 64-bit
definitions, elementwise within the bounds of plain64_gated.py, and by their
norms, in which a value left out would show."""
import numpy as np
import pytest

import plain64_gated as P
from test_gpu_linear_attn import DEV, _close, _np, _t

pytestmark = pytest.mark.gpu

# Rounding errors are 0.58 of half a step by the root of their mean square (a uniform one is 1 / sqrt(3)); a relative
# half step varies over a binade, so that 0.42 is usual; fp32 outputs carry a few dozen roundings, 4 U = 2.4e-7.
NORM = {"bf16": 1.2 * 2.0 ** -8 / np.sqrt(3), "f32": 1e-6}


def _compare(got, ref, types):
    for n, v in got.items():
        r, e = ref[n]
        r, e = r.reshape(v.shape), e.reshape(v.shape)
        _close(n, _np(v), r, P.tol(r, e, types[n]))
        if r.size > 100 and np.linalg.norm(r) > 0:
            assert np.linalg.norm(_np(v) - r) <= NORM[types[n]] * np.linalg.norm(r), n


def _wide(r, rows, D, dtype, pad):
    """(rows, D) values, rows D + pad apart, NaN between."""
    import torch
    v = _t(r.standard_normal((rows, D)), dtype)
    if pad == 0:
        return v
    w = torch.full((rows, D + pad), float("nan"), dtype=v.dtype, device=DEV)
    w[:, :D] = v
    return w[:, :D]


def _gated(seed, rows, D, groups, dtype, z=True, first=True, pad=0, eps=1e-6, w=True):
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(seed)
    x, zz = _wide(r, rows, D, dtype, pad), (_wide(r, rows, D, dtype, pad + pad // 2) if z else None)
    ww, dy = (_t(1 + 0.3 * r.standard_normal(D)) if w else None), _t(r.standard_normal((rows, D)), dtype)
    y = bd.ssm_gated_norm_fwd(x, zz, ww, groups=groups, gate_first=first, eps=eps)
    g = bd.ssm_gated_norm_bwd(x, zz, ww, dy=dy, groups=groups, gate_first=first, eps=eps)
    torch.cuda.synchronize()
    ref = P.gated_norm(_np(x), _np(zz), _np(ww), groups, first, eps, _np(dy))
    _compare({"y": y, **g}, ref, {"y": dtype, "dx": dtype, "dz": dtype, "dw": "f32"})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,groups", [(1, 1), (7, 1), (8, 1), (63, 3), (64, 8), (65, 1), (128, 1), (130, 2), (256, 1),
                                      (264, 1), (512, 1), (520, 1), (1001, 1), (1024, 8), (2048, 2), (2560, 1),
                                      (4100, 1), (5120, 1), (8192, 1), (8200, 1), (16384, 1), (16384, 2), (16383, 1)])
def test_gated_norm_widths(lib, D, groups, dtype):
    for first in (True, False):
        print("case", D, groups, dtype, first, flush=True)
        _gated(D + groups, 9, D, groups, dtype, first=first, pad=8 if D % 3 == 0 else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D,groups", [(1, 64, 1), (1, 5120, 1), (3, 96, 4), (700, 80, 1), (5000, 64, 2),
                                           (3001, 520, 1), (70001, 16, 1)])
def test_gated_norm_rows(lib, rows, D, groups, dtype):
    """One row to several rounds of every team."""
    print("case", rows, D, groups, dtype, flush=True)
    _gated(rows, rows, D, groups, dtype, first=rows % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 4, 8, 24])
def test_gated_norm_strides_and_options(lib, pad, dtype):
    print("case", pad, dtype, flush=True)
    _gated(pad, 33, 160, 2, dtype, pad=pad)
    _gated(pad, 33, 160, 1, dtype, z=False, pad=pad, eps=1e-2)
    _gated(pad, 33, 1000, 1, dtype, w=False, pad=pad, first=False)


def test_gated_norm_extremes(lib):
    """Gates shut and open to the limit, large and small rows, a group of zeros."""
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(1)
    x, z, dy = (_t(r.standard_normal((12, 96))) for _ in range(3))
    x[0] *= 1e15
    x[1] *= 1e-15
    x[2, :32] = 0
    z[3], z[4, ::2], z[5] = 90.0, -90.0, 0.0
    for first in (True, False):
        y = bd.ssm_gated_norm_fwd(x, z, None, groups=3, gate_first=first)
        g = bd.ssm_gated_norm_bwd(x, z, None, dy=dy, groups=3, gate_first=first)
        torch.cuda.synchronize()
        ref = P.gated_norm(_np(x), _np(z), None, 3, first, 1e-6, _np(dy))
        # dz of the row of 1e15 and of its reciprocal are compared with their own row's bounds; dw sums all rows.
        for n, v in {"y": y, **g}.items():
            _close(n, _np(v), ref[n][0], P.tol(*ref[n], "f32"))


def _residual(seed, rows, D, dtype, rt, post=True, pad=0, res=True, weights=True, alpha=0.7, eps=1e-6, tail=True):
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(seed)
    x = _wide(r, rows, D, dtype, pad)
    rr = _t(2 * r.standard_normal((rows, D)), rt) if res else None
    wp, wo = (_t(1 + 0.3 * r.standard_normal(D)) if weights else None for _ in range(2))
    dy, dR = _t(r.standard_normal((rows, D)), dtype), (_t(r.standard_normal((rows, D)), rt) if tail else None)
    import numpy
    al = float(numpy.float32(alpha))
    R, y = bd.ssm_residual_norm_fwd(x, rr, wp, wo, alpha=alpha, post_norm=post, eps=eps,
                                    res_dtype=torch.float32 if rt == "f32" else torch.bfloat16)
    g = bd.ssm_residual_norm_bwd(x, R, wp, wo, dy=dy, dres_out=dR, alpha=alpha, post_norm=post, eps=eps)
    torch.cuda.synchronize()
    _compare({"res_out": R, "y": y}, P.residual_norm(_np(x), _np(rr), _np(wp), _np(wo), al, post, eps),
             {"res_out": rt, "y": dtype})
    _compare(g, P.residual_norm_bwd(_np(x), _np(R), _np(wp), _np(wo), _np(dy), _np(dR), al, post, eps),
             {"dx": dtype, "dres": rt, "dw_pre": "f32", "dw_post": "f32"})


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("dtype,rt", TYPES)
@pytest.mark.parametrize("D", [1, 8, 60, 64, 100, 128, 256, 500, 512, 768, 1001, 2048, 2560, 5120, 8192, 8200, 16384])
def test_residual_norm_widths(lib, D, dtype, rt):
    for post in (True, False):
        print("case", D, dtype, rt, post, flush=True)
        _residual(D, 9, D, dtype, rt, post, pad=16 if D % 3 == 0 else 0)


@pytest.mark.parametrize("dtype,rt", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 64), (2, 2560), (1000, 72), (4100, 256), (3001, 520), (70001, 16)])
def test_residual_norm_rows(lib, rows, D, dtype, rt):
    print("case", rows, D, dtype, rt, flush=True)
    _residual(rows, rows, D, dtype, rt)


@pytest.mark.parametrize("dtype,rt", TYPES)
def test_residual_norm_options(lib, dtype, rt):
    _residual(1, 33, 160, dtype, rt, pad=5)
    _residual(2, 33, 160, dtype, rt, res=False, weights=False, tail=False, eps=1e-2)
    _residual(3, 33, 160, dtype, rt, post=False, alpha=0.0)
    _residual(4, 33, 161, dtype, rt, alpha=-2.5)


def test_outputs_in_place_and_given(lib):
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(5)
    for D in (96, 101, 1024, 5000):
        x, z, res, dy = (_t(r.standard_normal((2, 17, D)), "bf16") for _ in range(4))
        y = bd.ssm_gated_norm_fwd(x, z)
        R, n = bd.ssm_residual_norm_fwd(x, res, alpha=0.5)
        g = bd.ssm_residual_norm_bwd(x, R, dy=dy)
        k = bd.ssm_residual_norm_bwd(None, R, dy=dy, want_dw=False, want_dres=False, grads={"dx": torch.empty_like(x)})
        assert set(k) == {"dx"} and torch.equal(k["dx"], g["dx"]) and g["dx"].shape == x.shape
        k = bd.ssm_residual_norm_bwd(x, R, dy=dy, want_dw=False, grads={"dw_post": torch.empty(D, device=DEV)})
        assert set(k) == {"dx", "dres", "dw_post"} and torch.equal(k["dw_post"], g["dw_post"])
        got = bd.ssm_residual_norm_fwd(x, res, alpha=0.5, res_out=res)
        assert got[0] is res and torch.equal(res, R) and torch.equal(got[1], n)
        h = bd.ssm_gated_norm_bwd(x, z, dy=dy, want_dw=False)
        assert set(h) == {"dx", "dz"} and torch.equal(h["dx"], bd.ssm_gated_norm_bwd(x, z, dy=dy)["dx"])
        assert torch.equal(bd.ssm_gated_norm_fwd(x, z, y=x), y) and torch.equal(x, y)


def test_empty(lib):
    import torch
    from selective_state_space_84_amd import binding as bd
    x, w = torch.zeros(0, 64, device=DEV), torch.ones(64, device=DEV)
    assert bd.ssm_gated_norm_fwd(x, x, w).shape == (0, 64)
    assert not bd.ssm_gated_norm_bwd(x, x, w, dy=x)["dw"].any()
    R, y = bd.ssm_residual_norm_fwd(x, x, w)
    g = bd.ssm_residual_norm_bwd(x, R, w, w, dy=y)
    assert not g["dw_pre"].any() and not g["dw_post"].any()
    assert bd.ssm_gated_norm_fwd(torch.zeros(3, 0, device=DEV)).shape == (3, 0)


def test_large_offsets(lib):
    """More than 2^31 elements: the last rows against the same ones alone."""
    import torch
    from selective_state_space_84_amd import binding as bd
    n, D = 450001, 5120
    x = torch.empty(n, D, dtype=torch.bfloat16, device=DEV).normal_()
    y = bd.ssm_gated_norm_fwd(x, x)
    assert torch.equal(y[-5:], bd.ssm_gated_norm_fwd(x[-5:].clone(), x[-5:].clone()))
    g = bd.ssm_gated_norm_bwd(x, x, dy=y)
    k = bd.ssm_gated_norm_bwd(x[-5:].clone(), x[-5:].clone(), dy=y[-5:].clone())
    assert torch.equal(g["dx"][-5:], k["dx"]) and torch.equal(g["dz"][-5:], k["dz"])
    del g
    R, z = bd.ssm_residual_norm_fwd(x, y, post_norm=True)
    a = bd.ssm_residual_norm_fwd(x[-5:].clone(), y[-5:].clone(), post_norm=True)
    assert torch.equal(R[-5:], a[0]) and torch.equal(z[-5:], a[1])


def test_repeat_stream_and_graph(lib):
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(6)
    x, z, dy = (_t(r.standard_normal((900, 320)), "bf16") for _ in range(3))
    res = _t(r.standard_normal((900, 320)))
    w = _t(r.standard_normal(320))

    def step(stream=None):
        y = bd.ssm_gated_norm_fwd(x, z, w, groups=5, stream=stream)
        R, n = bd.ssm_residual_norm_fwd(y, res, w, w, post_norm=True, stream=stream)
        g = bd.ssm_residual_norm_bwd(y, R, w, w, dy=dy, post_norm=True, stream=stream)
        k = bd.ssm_gated_norm_bwd(x, z, w, dy=g["dx"], groups=5, stream=stream)
        return [y, R, n, *g.values(), *k.values()]
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        dy.mul_(1.5)
        want = step()
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), i
