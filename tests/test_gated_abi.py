"""Argument checks of the gated recurrence, the gated norm and the residual norm
(nothing is launched): on the host, before any memory is touched."""
import ctypes

import pytest

from selective_state_space_84_amd import binding as bd

P0 = 0x7F0000000000
MB = 1 << 20
BAD = ctypes.c_size_t(-1).value


def _fwd(lib, x=P0, ga=P0 + MB, gx=P0 + 2 * MB, la=P0 + 3 * MB, z=None, lens=None, h0=None, y=P0 + 4 * MB, hl=None,
         ck=None, b=2, L=40, D=96, xs=0, as_=0, is_=0, zs=0, dtype=1, ws=P0 + 90 * MB, wsb=MB):
    return lib.ssm_gated_scan_fwd(x, ga, gx, la, z, lens, h0, y, hl, ck, b, L, D, xs, as_, is_, zs, dtype, ws, wsb,
                                  None)


def test_scan_errors(lib):
    for name in ("x", "ga", "gx", "la", "y"):
        assert _fwd(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    assert _fwd(lib, L=0, la=None) == bd.SSM_ERR_NULL_ARG
    for bad in (dict(b=-1), dict(L=-1), dict(D=-1), dict(L=(1 << 31) - 100), dict(D=(1 << 23) + 1),
                dict(b=1 << 40, L=1 << 20), dict(b=1 << 20, D=1 << 12), dict(xs=95), dict(zs=8, z=P0 + 5 * MB),
                dict(as_=(1 << 25) + 1), dict(b=1 << 62, D=1), dict(is_=1 << 25, b=1 << 20, L=1 << 20, D=1),
                dict(b=1 << 20, L=1 << 20, D=1)):
        assert _fwd(lib, **bad) == bd.SSM_ERR_BAD_DIM, bad
    assert _fwd(lib, dtype=2) == bd.SSM_ERR_UNSUPPORTED
    for name, p in (("x", P0), ("ga", P0 + MB), ("gx", P0 + 2 * MB), ("z", P0 + 5 * MB), ("y", P0 + 4 * MB)):
        assert _fwd(lib, **{name: p + 1}) == bd.SSM_ERR_MISALIGNED, name
        assert _fwd(lib, **{name: p + 2, "dtype": 0}) == bd.SSM_ERR_MISALIGNED, name
    for name in ("la", "lens", "h0", "hl", "ck"):
        assert _fwd(lib, **{name: P0 + 6 * MB + 2}) == bd.SSM_ERR_MISALIGNED, name
    for bad in (dict(y=P0 + 64), dict(y=P0 + MB), dict(hl=P0 + 2 * MB), dict(ck=P0 + 4 * MB),
                dict(h0=P0 + 7 * MB, hl=P0 + 7 * MB + 4), dict(h0=P0 + 4 * MB, hl=P0 + 4 * MB),
                dict(h0=P0 + 7 * MB, ck=P0 + 7 * MB), dict(z=P0 + 4 * MB), dict(y=P0 + 3 * MB)):
        assert _fwd(lib, **bad) == bd.SSM_ERR_ALIAS, bad


def test_scan_workspace(lib):
    need = lib.ssm_gated_scan_fwd_workspace_size(2, 4096, 96, 1)
    assert need % 4 == 0 and need < MB
    if need:
        assert _fwd(lib, L=4096, ws=None) == bd.SSM_ERR_WORKSPACE
        assert _fwd(lib, L=4096, wsb=need - 1) == bd.SSM_ERR_WORKSPACE
        assert _fwd(lib, L=4096, ws=P0 + 90 * MB + 128) == bd.SSM_ERR_MISALIGNED
        assert _fwd(lib, L=4096, ws=P0 + 4 * MB) == bd.SSM_ERR_ALIAS
        assert _fwd(lib, L=4096, ws=P0 + 256) == bd.SSM_ERR_ALIAS
        assert _fwd(lib, L=4096, h0=P0 + 90 * MB, hl=P0 + 90 * MB) == bd.SSM_ERR_ALIAS
    assert lib.ssm_gated_scan_ckpt_bytes(2, 65, 96) == lib.ssm_gated_scan_ckpt_bytes(2, 128, 96)
    assert lib.ssm_gated_scan_ckpt_bytes(2, 0, 96) == 0
    for args in ((-1, 4, 4), (1, -1, 4), (1, 4, 1 << 24), (1 << 30, 4, 1 << 22)):
        assert lib.ssm_gated_scan_fwd_workspace_size(*args, 1) == BAD
        assert lib.ssm_gated_scan_bwd_workspace_size(*args, 1, 0) == BAD
        assert lib.ssm_gated_scan_ckpt_bytes(*args) == BAD
    assert lib.ssm_gated_scan_fwd_workspace_size(1, 4, 4, 7) == BAD
    assert lib.ssm_gated_scan_bwd_workspace_size(1, 4, 4, 1, 2) == BAD
    assert lib.ssm_gated_scan_bwd_workspace_size(2, 4096, 96, 1, 1) <= lib.ssm_gated_scan_bwd_workspace_size(
        2, 4096, 96, 1, 0)


def test_scan_pieces_stay_countable(lib):
    """Pieces of 64 steps and 64 channels are counted in 31 bits; workspaces of large calls stay exact in 64."""
    for args, ok in (((1, 1, 1 << 23), True), ((16384, 64, 1 << 23), False), ((1, (1 << 31) - 257, 64), True),
                     ((65, (1 << 31) - 257, 64), False), ((64, (1 << 31) - 257, 64), True),
                     (((1 << 31), 1, 1), False), (((1 << 31) - 1, 1, 1), True), (((1 << 24), 64 * 128, 1), False)):
        for f in (lambda *a: lib.ssm_gated_scan_fwd_workspace_size(*a, 1),
                  lambda *a: lib.ssm_gated_scan_bwd_workspace_size(*a, 0, 0), lib.ssm_gated_scan_ckpt_bytes):
            assert (f(*args) != BAD) == ok, args
    b, L, D = 63, (1 << 31) - 257, 64
    pieces = -(-L // 128)
    assert lib.ssm_gated_scan_fwd_workspace_size(b, L, D, 1) >= b * D * pieces * 8
    assert lib.ssm_gated_scan_ckpt_bytes(b, L, D) == b * D * -(-L // 64) * 4
    assert lib.ssm_gated_scan_fwd_workspace_size(8, 128, 64, 1) == 0
    # A call of one piece needs no workspace; one of two does.
    assert lib.ssm_gated_scan_fwd_workspace_size(8, 129, 64, 1) > 0


def test_scan_empty(lib):
    """Calls without an element or a state launch nothing."""
    assert _fwd(lib, b=0, x=None, ga=None, gx=None, la=None, y=None) == bd.SSM_OK
    assert _fwd(lib, D=0, x=None, ga=None, gx=None, la=None, y=None) == bd.SSM_OK


def test_counts_without_an_element(lib):
    """Rows and groups of nothing are still counted in 64 bits, also in bytes."""
    for b in (1 << 62, (1 << 48) + 1):
        assert _fwd(lib, b=b, L=0, D=0, lens=P0 + 6 * MB) == bd.SSM_ERR_BAD_DIM
        assert _bwd(lib, b=b, L=0, D=0, lens=P0 + 6 * MB) == bd.SSM_ERR_BAD_DIM
        assert lib.ssm_gated_scan_fwd_workspace_size(b, 0, 0, 1) == BAD
    assert _fwd(lib, b=1 << 48, L=0, D=0) == bd.SSM_OK
    for groups in ((1 << 62) + 1, (1 << 23) + 1):
        assert lib.ssm_gated_norm_fwd(P0, None, None, P0 + MB, 4, 0, groups, 0, 0, 1e-6, 1, 1, None) == \
            bd.SSM_ERR_BAD_DIM
        assert lib.ssm_gated_norm_bwd(P0, None, None, P0 + MB, P0 + 2 * MB, None, P0 + 3 * MB, 4, 0, groups, 0, 0, 1e-6,
                                      1, 1, P0 + 4 * MB, MB, None) == bd.SSM_ERR_BAD_DIM
        assert lib.ssm_gated_norm_bwd_workspace_size(4, 0, groups) == BAD
    assert lib.ssm_gated_norm_fwd(P0, None, None, P0 + MB, 4, 0, 1 << 23, 0, 0, 1e-6, 1, 1, None) == bd.SSM_OK


def _bwd(lib, x=P0, ga=P0 + MB, gx=P0 + 2 * MB, la=P0 + 3 * MB, z=None, lens=None, h0=None, dy=P0 + 4 * MB, dh=None,
         ck=None, dx=P0 + 10 * MB, dga=P0 + 11 * MB, dgx=P0 + 12 * MB, dz=None, dla=P0 + 13 * MB, dh0=None, b=2, L=40,
         D=96, xs=0, dtype=1, ws=P0 + 90 * MB, wsb=8 * MB):
    return lib.ssm_gated_scan_bwd(x, ga, gx, la, z, lens, h0, dy, dh, ck, dx, dga, dgx, dz, dla, dh0, b, L, D, xs, 0, 0,
                                  0, dtype, ws, wsb, None)


def test_scan_gradient_errors(lib):
    for name in ("x", "ga", "gx", "la", "dy", "dx", "dga", "dgx"):
        assert _bwd(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    assert _bwd(lib, z=P0 + 5 * MB) == bd.SSM_ERR_NULL_ARG
    assert _bwd(lib, dz=P0 + 5 * MB) == bd.SSM_ERR_NULL_ARG
    assert _bwd(lib, xs=90) == bd.SSM_ERR_BAD_DIM
    assert _bwd(lib, dtype=-1) == bd.SSM_ERR_UNSUPPORTED
    for name in ("dx", "dga", "dgx", "dy"):
        assert _bwd(lib, **{name: P0 + 20 * MB + 1}) == bd.SSM_ERR_MISALIGNED, name
    for name in ("dla", "dh0", "ck", "dh"):
        assert _bwd(lib, **{name: P0 + 20 * MB + 2}) == bd.SSM_ERR_MISALIGNED, name
    for bad in (dict(dx=P0), dict(dga=P0 + 10 * MB), dict(dgx=P0 + 4 * MB), dict(dla=P0 + 3 * MB),
                dict(h0=P0 + 6 * MB, dh0=P0 + 6 * MB), dict(dh=P0 + 6 * MB, dh0=P0 + 6 * MB),
                dict(ck=P0 + 6 * MB, dh0=P0 + 6 * MB), dict(ws=P0 + 10 * MB), dict(ws=P0 + 4 * MB),
                dict(h0=P0 + 90 * MB)):
        assert _bwd(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    need = lib.ssm_gated_scan_bwd_workspace_size(2, 40, 96, 1, 0)
    assert need > 0
    assert _bwd(lib, wsb=need - 1) == bd.SSM_ERR_WORKSPACE
    assert _bwd(lib, ws=None) == bd.SSM_ERR_WORKSPACE
    assert _bwd(lib, ws=P0 + 90 * MB + 4) == bd.SSM_ERR_MISALIGNED
    assert _bwd(lib, D=0) == bd.SSM_OK


def _upd(lib, h=P0, slots=None, x=P0 + MB, ga=P0 + 2 * MB, gx=P0 + 3 * MB, la=P0 + 4 * MB, z=None, y=P0 + 5 * MB, b=4,
         n=4, D=96, xs=0, zs=0, dtype=1):
    return lib.ssm_gated_scan_update(h, slots, x, ga, gx, la, z, y, b, n, D, xs, 0, 0, zs, dtype, None)


def test_update_errors(lib):
    for name in ("h", "x", "ga", "gx", "la", "y"):
        assert _upd(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    for bad in (dict(b=-1), dict(n=-1), dict(D=-1), dict(n=5), dict(xs=95), dict(z=P0 + 7 * MB, zs=95),
                dict(xs=(1 << 40) + 1), dict(D=(1 << 23) + 1), dict(b=1 << 24, n=1 << 24, D=1),
                dict(b=1 << 20, n=1 << 20, D=8192)):
        assert _upd(lib, **bad) == bd.SSM_ERR_BAD_DIM, bad
    assert _upd(lib, dtype=3) == bd.SSM_ERR_UNSUPPORTED
    for name in ("x", "ga", "gx", "z", "y"):
        assert _upd(lib, **{name: P0 + 8 * MB + 1}) == bd.SSM_ERR_MISALIGNED, name
    for name in ("h", "slots", "la"):
        assert _upd(lib, **{name: P0 + 8 * MB + 2}) == bd.SSM_ERR_MISALIGNED, name
    for bad in (dict(y=P0), dict(y=P0 + MB), dict(h=P0 + 4 * MB), dict(slots=P0), dict(z=P0 + 5 * MB)):
        assert _upd(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    assert _upd(lib, b=0, n=7, slots=P0 + 9 * MB) == bd.SSM_OK


def _gn(lib, x=P0, z=P0 + MB, w=P0 + 2 * MB, y=P0 + 3 * MB, rows=8, D=96, G=1, xs=0, zs=0, eps=1e-6, first=1, dtype=1):
    return lib.ssm_gated_norm_fwd(x, z, w, y, rows, D, G, xs, zs, eps, first, dtype, None)


def _gnb(lib, x=P0, z=P0 + MB, w=P0 + 2 * MB, dy=P0 + 3 * MB, dx=P0 + 4 * MB, dz=P0 + 5 * MB, dw=P0 + 6 * MB, rows=8,
         D=96, G=1, xs=0, zs=0, eps=1e-6, first=1, dtype=1, ws=P0 + 90 * MB, wsb=MB):
    return lib.ssm_gated_norm_bwd(x, z, w, dy, dx, dz, dw, rows, D, G, xs, zs, eps, first, dtype, ws, wsb, None)


def test_gated_norm_errors(lib):
    for f in (_gn, _gnb):
        assert f(lib, x=None) == bd.SSM_ERR_NULL_ARG
        for bad in (dict(rows=-1), dict(D=-1), dict(G=0), dict(G=-2), dict(xs=95), dict(zs=95), dict(rows=1 << 48),
                    dict(D=(1 << 23) + 8, G=1 << 20)):
            assert f(lib, **bad) == bd.SSM_ERR_BAD_DIM, bad
        for bad in (dict(G=5), dict(D=16392), dict(eps=-1.0), dict(eps=float("nan")), dict(first=2), dict(dtype=9)):
            assert f(lib, **bad) == bd.SSM_ERR_UNSUPPORTED, bad
        for name in ("x", "z"):
            assert f(lib, **{name: P0 + 20 * MB + 1}) == bd.SSM_ERR_MISALIGNED, name
        assert f(lib, w=P0 + 20 * MB + 2) == bd.SSM_ERR_MISALIGNED
    assert _gn(lib, y=None) == bd.SSM_ERR_NULL_ARG
    for bad in (dict(y=P0 + 2), dict(y=P0 + MB), dict(y=P0 + 2 * MB), dict(y=P0, xs=128)):
        assert _gn(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    assert _gn(lib, rows=0, x=None, y=None) == bd.SSM_OK
    for name in ("dy", "dx", "dz"):
        assert _gnb(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    assert _gnb(lib, z=None) == bd.SSM_ERR_NULL_ARG
    for bad in (dict(dx=P0), dict(dz=P0 + 4 * MB), dict(dw=P0 + 2 * MB), dict(dx=P0 + 3 * MB), dict(ws=P0),
                dict(ws=P0 + 5 * MB)):
        assert _gnb(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    need = lib.ssm_gated_norm_bwd_workspace_size(8, 96, 1)
    assert 0 < need <= MB
    assert _gnb(lib, wsb=need - 1) == bd.SSM_ERR_WORKSPACE
    assert _gnb(lib, ws=None) == bd.SSM_ERR_WORKSPACE
    assert _gnb(lib, ws=P0 + 90 * MB + 8) == bd.SSM_ERR_MISALIGNED
    assert lib.ssm_gated_norm_bwd_workspace_size(0, 96, 1) == 0
    for args in ((-1, 96, 1), (8, 96, 5), (8, 16400, 1), (8, 96, 0)):
        assert lib.ssm_gated_norm_bwd_workspace_size(*args) == BAD, args


def _rn(lib, x=P0, res=P0 + MB, wp=P0 + 2 * MB, wo=P0 + 3 * MB, out=P0 + 4 * MB, y=P0 + 5 * MB, rows=8, D=96, xs=0,
        alpha=1.0, eps=1e-6, post=1, dtype=1, rd=0):
    return lib.ssm_residual_norm_fwd(x, res, wp, wo, out, y, rows, D, xs, alpha, eps, post, dtype, rd, None)


def _rnb(lib, x=P0, out=P0 + MB, wp=P0 + 2 * MB, wo=P0 + 3 * MB, dy=P0 + 4 * MB, dout=P0 + 5 * MB, dx=P0 + 6 * MB,
         dres=P0 + 7 * MB, dwp=P0 + 8 * MB, dwo=P0 + 9 * MB, rows=8, D=96, xs=0, alpha=1.0, eps=1e-6, post=1, dtype=1,
         rd=0, ws=P0 + 90 * MB, wsb=MB):
    return lib.ssm_residual_norm_bwd(x, out, wp, wo, dy, dout, dx, dres, dwp, dwo, rows, D, xs, alpha, eps, post, dtype,
                                     rd, ws, wsb, None)


def test_residual_norm_errors(lib):
    for f in (_rn, _rnb):
        assert f(lib, x=None) == bd.SSM_ERR_NULL_ARG
        for bad in (dict(rows=-1), dict(D=-1), dict(xs=95), dict(rows=1 << 47)):
            assert f(lib, **bad) == bd.SSM_ERR_BAD_DIM, bad
        for bad in (dict(D=16385), dict(eps=-1.0), dict(post=2), dict(post=-1), dict(dtype=2), dict(rd=2),
                    dict(dtype=0, rd=1)):
            assert f(lib, **bad) == bd.SSM_ERR_UNSUPPORTED, bad
        for name, p in (("x", 1), ("wp", 2), ("wo", 2), ("out", 2)):
            assert f(lib, **{name: P0 + 20 * MB + p}) == bd.SSM_ERR_MISALIGNED, name
    for name in ("out", "y"):
        assert _rn(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    for bad in (dict(out=P0), dict(y=P0 + MB), dict(y=P0 + 4 * MB), dict(out=P0 + MB + 4), dict(y=P0 + 3 * MB)):
        assert _rn(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    assert _rn(lib, rows=0, x=None, out=None, y=None) == bd.SSM_OK
    for name in ("out", "dy", "dx"):
        assert _rnb(lib, **{name: None}) == bd.SSM_ERR_NULL_ARG, name
    assert _rnb(lib, x=None, post=0) == bd.SSM_ERR_NULL_ARG
    for bad in (dict(dx=P0 + 4 * MB), dict(dres=P0 + 5 * MB), dict(dres=P0 + 6 * MB), dict(dwo=P0 + 8 * MB),
                dict(ws=P0 + 7 * MB), dict(dx=P0)):
        assert _rnb(lib, **bad) == bd.SSM_ERR_ALIAS, bad
    need = lib.ssm_residual_norm_bwd_workspace_size(8, 96)
    assert 0 < need <= MB
    assert _rnb(lib, wsb=need - 1) == bd.SSM_ERR_WORKSPACE
    assert _rnb(lib, ws=P0 + 90 * MB + 16) == bd.SSM_ERR_MISALIGNED
    assert lib.ssm_residual_norm_bwd_workspace_size(-1, 96) == BAD
    assert lib.ssm_residual_norm_bwd_workspace_size(8, 16385) == BAD


def test_binding_refusals():
    """Shapes and types that do not fit are named before anything reaches the library."""
    import torch
    x = torch.zeros(2, 5, 8)
    la = torch.zeros(8)
    for bad in (dict(ga=torch.zeros(2, 5, 7)), dict(gx=torch.zeros(2, 5, 8).bfloat16()), dict(log_a=torch.zeros(7)),
                dict(z=torch.zeros(2, 4, 8)), dict(lengths=torch.zeros(2)), dict(h0=torch.zeros(2, 7)),
                dict(x=torch.zeros(5, 8)), dict(x=x.double())):
        with pytest.raises(ValueError):
            bd.ssm_gated_scan_fwd(**{**dict(x=x, ga=x, gx=x, log_a=la), **bad})
    with pytest.raises(ValueError, match="dy"):
        bd.ssm_gated_scan_bwd(x, x, x, la, dy=torch.zeros(2, 5, 7))
    with pytest.raises(ValueError, match="h must"):
        bd.ssm_gated_scan_update(torch.zeros(4, 7), x[:, 0], x[:, 0], x[:, 0], la)
    with pytest.raises(ValueError, match="w must"):
        bd.ssm_gated_norm_fwd(x, None, torch.zeros(7))
    with pytest.raises(ValueError, match="residual"):
        bd.ssm_residual_norm_fwd(x, torch.zeros(2, 5, 7))
    with pytest.raises(ValueError, match="residual"):
        bd.ssm_residual_norm_fwd(x, x.half())
    with pytest.raises(ValueError, match="GPU"):
        bd.ssm_gated_norm_fwd(x)


class _View:
    """What _steps looks at, without a GPU."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, n):
        return getattr(self.t, n)


def test_binding_rows(lib):
    import torch
    w = torch.zeros(3, 4, 20)
    assert bd._steps(_View(w), "x")[1] == 20
    p, step = bd._steps(_View(w[:, :, 4:12]), "x")
    assert step == 20 and p == w.data_ptr() + 16
    assert bd._steps(_View(w[:, 1:2, :8]), "x")[1] == 80
    assert bd._steps(_View(w[1:2, 2:3, :8]), "x")[1] == 8
    assert bd._steps(_View(w[:, 0]), "x")[1] == 80
    for bad in (w[:, :2], w[:, :, ::2], w.transpose(0, 1), w[:1, :1].expand(3, 4, 20), w.transpose(1, 2)):
        with pytest.raises(ValueError, match="rows"):
            bd._steps(_View(bad), "x")
