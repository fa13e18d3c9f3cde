"""Calls of the gated recurrence in every combination of what may be given and
left out, and chains of pieces in blocks of both lengths that rows end in,
against the 64-bit definitions within the bounds of plain64_gated.py."""
import numpy as np
import pytest

import plain64_gated as P
from test_gpu_gated_scan import _lens, _make
from test_gpu_linear_attn import _close, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(40))
def test_any_call(lib, seed):
    """Sizes, types, strides, options and row lengths at random; what is behind a row's end is NaN."""
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(100 + seed)
    flag = lambda: bool(r.integers(2))  # noqa: E731
    dtype, B, D = ("f32", "bf16")[r.integers(2)], int(r.integers(1, 6)), int(np.exp(r.uniform(0, 5.2)))
    L = int(np.exp(r.uniform(0, 6.8)))
    z, h0, dh_last, ckpt, dh0, dlog_a = (flag() for _ in range(6))
    d, dy, dh = _make(seed, B, L, D, dtype, z=z, fused=flag(), pad=int(r.integers(0, 5)))
    if not h0:
        d["h0"] = None
    if not dh_last:
        dh = None
    lengths = None
    if flag():
        lengths = [int(v) for v in r.integers(-1, L + 2, B)]
        for b, n in enumerate(lengths):
            for t in (d["x"], d["ga"], d["gx"], d["z"], dy):
                if t is not None:
                    t[b, max(n, 0):] = float("nan")
    print("case", dtype, B, L, D, z, h0, dh_last, ckpt, dh0, dlog_a, lengths, flush=True)
    y, hl, ck = bd.ssm_gated_scan_fwd(**d, lengths=_lens(lengths), want_ckpt=ckpt)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, lengths=_lens(lengths), dh_last=dh, ckpt=ck, want_dh0=dh0,
                              want_dlog_a=dlog_a)
    torch.cuda.synchronize()
    assert ("dh0" in g) == dh0 and ("dlog_a" in g) == dlog_a and ("dz" in g) == z
    ref = P.scan(**{k: _np(v) for k, v in d.items()}, lengths=lengths, dy=_np(dy), dh_last=_np(dh))
    for n, v in {"y": y, "h_last": hl, **g}.items():
        _close(n, _np(v), ref[n][0], P.tol(*ref[n], "f32" if n in ("h_last", "dlog_a", "dh0") else dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [16, 900])
def test_long_padded_batch(lib, D, dtype):
    """Rows that end in every kind of piece and block of a long chain: few chains, whose blocks have 32 pieces (4096
    steps forward, 2048 back), and many, whose blocks have 8; the last state in place of the first."""
    import torch
    from selective_state_space_84_amd import binding as bd
    L = 9000
    lengths = [L, 4096, 4097, 2049, 0, 8191, 6145]
    d, dy, dh = _make(D, len(lengths), L, D, dtype, log_a=-np.exp(np.random.default_rng(1).uniform(-9, 0, D)))
    cut = np.linspace(0, D - 1, 16).astype(int)  # the channels that are compared
    for b, n in enumerate(lengths):
        for t in (d["x"], d["ga"], d["gx"], d["z"], dy):
            t[b, n:] = float("nan")
    y, hl, ck = bd.ssm_gated_scan_fwd(**d, lengths=_lens(lengths), want_ckpt=True)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, lengths=_lens(lengths), dh_last=dh, ckpt=ck)
    again = bd.ssm_gated_scan_bwd(**d, dy=dy, lengths=_lens(lengths), dh_last=dh)
    h = d["h0"].clone()
    y2, h2, _ = bd.ssm_gated_scan_fwd(**{**d, "h0": h}, lengths=_lens(lengths), h_last=h)
    torch.cuda.synchronize()
    assert h2 is h and torch.equal(h, hl) and torch.equal(y2, y)
    assert all(torch.equal(again[k], g[k]) for k in g)
    for n, v in {"y": y, **{k: g[k] for k in ("dx", "dga", "dgx", "dz")}}.items():
        for b, k in enumerate(lengths):
            assert not v[b, k:].any() and torch.isfinite(v[b, :k]).all(), (n, b)
    ins = {k: _np(v[..., cut]) for k, v in d.items()}
    ref = P.scan(**ins, lengths=lengths, dy=_np(dy[..., cut]), dh_last=_np(dh[..., cut]))
    for n, v in {"y": y, "h_last": hl, **g}.items():
        _close(n, _np(v[..., cut]), ref[n][0], P.tol(*ref[n], "f32" if n in ("h_last", "dlog_a", "dh0") else dtype))
