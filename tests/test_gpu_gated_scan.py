"""Gated recurrence (whole sequences, gradient, one step) against the 64-bit
definitions, elementwise within the bounds of plain64_gated.py."""
import numpy as np
import pytest

import plain64_gated as P
from test_gpu_linear_attn import DEV, _close, _np, _t

pytestmark = pytest.mark.gpu


def _make(seed, B, L, D, dtype, z=True, states=True, fused=True, log_a=None, pad=2):
    """Inputs on the device; fused: the gates are column ranges of one wider tensor, `pad` columns apart.  (bf16 rows of
    even widths and distances are read in pairs, others one by one.)"""
    r = np.random.default_rng(seed)
    parts = [_t(1.5 * r.standard_normal((B, L, D)), dtype) for _ in range(3 if z else 2)]
    if fused:
        import torch
        wide = torch.full((B, L, len(parts) * (D + pad)), float("nan"), dtype=parts[0].dtype, device=DEV)
        for i, p in enumerate(parts):
            wide[:, :, i * (D + pad):i * (D + pad) + D] = p
            parts[i] = wide[:, :, i * (D + pad):i * (D + pad) + D]
    if log_a is None:
        log_a = -np.exp(r.uniform(-4.6, 1.4, D))
    d = dict(x=_t(r.standard_normal((B, L, D)), dtype), ga=parts[0], gx=parts[1], z=parts[2] if z else None,
             log_a=_t(np.asarray(log_a)), h0=_t(r.standard_normal((B, D))) if states else None)
    dy = _t(r.standard_normal((B, L, D)), dtype)
    dh = _t(r.standard_normal((B, D))) if states else None
    return d, dy, dh


def _lens(lengths):
    import torch
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)


def _check(d, dy, dh, dtype, lengths=None, ckpt=True):
    """Forward and gradient of one call, with saved states and without."""
    import torch
    from selective_state_space_84_amd import binding as bd
    ins = {k: _np(v) for k, v in d.items()}
    ref = P.scan(**ins, lengths=lengths, dy=_np(dy), dh_last=_np(dh))
    y, hl, ck = bd.ssm_gated_scan_fwd(**d, lengths=_lens(lengths), want_ckpt=True)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, lengths=_lens(lengths), dh_last=dh, ckpt=ck if ckpt else None)
    torch.cuda.synchronize()
    assert set(g) == {"dx", "dga", "dgx", "dlog_a", "dh0"} | ({"dz"} if d["z"] is not None else set())
    got = {"y": y, "h_last": hl, **g}
    for n, v in got.items():
        _close(n, _np(v), ref[n][0], P.tol(*ref[n], "f32" if n in ("h_last", "dlog_a", "dh0") else dtype))
        if n in ("y", "dx", "dga", "dgx", "dz") and lengths is not None:
            for b, k in enumerate(lengths):
                assert not v[b, max(k, 0):].any(), (n, b)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1025])
def test_lengths(lib, L, dtype):
    for D in (70, 71):
        print("case", L, D, dtype, flush=True)
        _check(*_make(L, 2, L, D, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("D", [1, 2, 3, 63, 64, 65, 127, 128, 130, 257, 512])
def test_widths(lib, D, z, dtype):
    print("case", D, z, dtype, flush=True)
    _check(*_make(D, 2, 150, D, dtype, z=z, states=z, fused=D % 2 == 1), dtype, ckpt=z)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 2, 8])
def test_strides(lib, pad, dtype):
    """Rows at odd distances, and at even ones with the width odd and even."""
    for D in (64, 129):
        print("case", D, pad, dtype, flush=True)
        _check(*_make(pad, 2, 140, D, dtype, pad=pad), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("lengths", [None, [700, 0, 699, 129, 1]])
def test_rows_of_whole_cache_lines(lib, lengths, z, dtype):
    """Rows of 128 bytes and multiples, also as column ranges, which the caches are told about: the definition's
    results, and to the bit those of the same rows elsewhere in memory; with and without saved states."""
    import torch
    from selective_state_space_84_amd import binding as bd
    B, L = 5, 700
    for D, pad in ((64, 64), (192, 0)):
        print("case", D, pad, flush=True)
        d, dy, dh = _make(D, B, L, D, dtype, z=z, pad=pad)
        if lengths is not None:
            for b, n in enumerate(lengths):
                for t in (d["x"], d["ga"], d["gx"], d["z"], dy):
                    if t is not None:
                        t[b, n:] = float("nan")
        got = _check(d, dy, dh, dtype, lengths)
        other = dict(d)
        for k in ("x", "ga", "gx", "z"):
            if d[k] is not None:
                wide = torch.empty(B, L, D + 2, dtype=d[k].dtype, device=DEV)
                other[k] = wide[:, :, :D].copy_(d[k])
        for ins in (d, other):
            y, hl, none = bd.ssm_gated_scan_fwd(**ins, lengths=_lens(lengths))
            assert none is None and torch.equal(y, got["y"]) and torch.equal(hl, got["h_last"])
            g = bd.ssm_gated_scan_bwd(**ins, dy=dy, lengths=_lens(lengths), dh_last=dh)
            for k, v in g.items():
                assert torch.equal(v, got[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("L,lengths,D", [
    (400, [400, 399, 0, 1, 128, 129, 64, 257, -3], 100),
    (400, [33, 400, 15, 16, 17], 101),
    (2600, [2600, 2599, 511, 512, 513, 576, 577, 1023, 1024, 1025, 1152, 0, 2048, 2049, 63, 1600], 20),
])
def test_padded_batch(lib, L, lengths, D, ckpt, dtype):
    """Rows that end anywhere, also at and beyond both ends; NaN behind them reaches nothing."""
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(5, len(lengths), L, D, dtype)
    for b, n in enumerate(lengths):
        for t in (d["x"], d["ga"], d["gx"], d["z"], dy):
            t[b, max(n, 0):] = float("nan")
    got = _check(d, dy, dh, dtype, lengths, ckpt)
    again = bd.ssm_gated_scan_fwd(**d, lengths=_lens([n + 1000 if n == L else n for n in lengths]))
    assert torch.equal(again[0], got["y"]) and torch.equal(again[1], got["h_last"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_extremes(lib, dtype):
    """Channels that forget nothing, hardly anything, and everything at once; gates shut and open to the limit."""
    import torch
    D = 96
    log_a = np.array([0.0, -1e-30, -1e-12, -1e-7, -1e-5, -80.0, -200.0, -1e4] * 12, dtype=np.float32)
    d, dy, dh = _make(6, 2, 200, D, dtype, log_a=log_a)
    for i, v in enumerate((100.0, -100.0, 40.0, -40.0)):
        d["ga"][:, i::7] = v
        d["gx"][:, i + 1::9] = -v
        d["z"][:, i + 2::11] = v
    ins = {k: _np(v) for k, v in d.items()}
    m2 = -np.expm1(2 * ins["log_a"] * P.sigmoid(ins["ga"]))
    assert not ((m2 > 0.9 * P.TINY) & (m2 < 1.1 * P.TINY)).any()  # on one side of the border of what counts
    from selective_state_space_84_amd import binding as bd
    ref = P.scan(**ins, dy=_np(dy), dh_last=_np(dh))
    y, hl, ck = bd.ssm_gated_scan_fwd(**d, want_ckpt=True)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck)
    torch.cuda.synchronize()
    for n, v in {"y": y, "h_last": hl, **g}.items():
        _close(n, _np(v), ref[n][0], P.tol(*ref[n], "f32" if n in ("h_last", "dlog_a", "dh0") else dtype))


def test_non_finite_values_stay_in_their_channel(lib):
    """A NaN or an infinity reaches the later steps of its row and channel, and nothing else."""
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(7, 2, 600, 70, "bf16")
    want = bd.ssm_gated_scan_fwd(**d)[0]
    d["x"][0, 200, 10] = float("inf")
    d["ga"][1, 300, 20] = float("nan")
    got = bd.ssm_gated_scan_fwd(**d)[0]
    same = torch.ones_like(want, dtype=torch.bool)
    same[0, 200:, 10] = False
    same[1, 300:, 20] = False
    assert torch.equal(got[same], want[same])
    assert not torch.isfinite(got[0, 200, 10]) and torch.isnan(got[1, 300:, 20]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(1, 5000, 200), (3, 2100, 64), (1, 9000, 2), (40, 520, 130), (2, 1500, 33)])
def test_long_sequences(lib, B, L, D, dtype):
    """States handed on many times, few and many channels; small errors by the outputs' norms too."""
    d, dy, dh = _make(B + L, B, L, D, dtype)
    print("case", B, L, D, dtype, flush=True)
    got = _check(d, dy, dh, dtype, ckpt=B != 3)
    ref = P.scan(**{k: _np(v) for k, v in d.items()}, dy=_np(dy), dh_last=_np(dh))
    # A step's decay is off by 2 U of the hardware's exponential (which leans to one side), log_a's roundings times
    # |log a|, and 3 roundings, 5.5 U together for slow channels; errors that lean add up over what a state remembers,
    # T = 1 / (1 - a) steps with the gate half open: 5.5 U T for a state or a state's gradient, twice that for their
    # product.
    T = 1.0 / (1.0 - np.exp(0.5 * float(d["log_a"].max())))
    for n, lim in (("h_last", 5.5), ("dh0", 5.5), ("dlog_a", 11.0), ("y", 5.5), ("dx", 5.5), ("dgx", 5.5),
                   ("dga", 11.0), ("dz", 5.5)):
        half = 1.2 * 2.0 ** -8 / np.sqrt(3) if dtype == "bf16" and got[n].dim() == 3 else 0.0
        err = np.linalg.norm(_np(got[n]) - ref[n][0]) / np.linalg.norm(ref[n][0])
        print("  %s by its norm: %.2g" % (n, err), flush=True)
        assert err <= half + lim * P.U * T, n


def test_options(lib):
    """Without states, lengths, saved states or sums, outputs given, and in place of h0."""
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(8, 2, 333, 72, "bf16")
    y, hl, none = bd.ssm_gated_scan_fwd(**d)
    assert none is None
    buf, h = torch.empty_like(y), d["h0"].clone()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = bd.ssm_gated_scan_fwd(**{**d, "h0": h}, y=buf, h_last=h, workspace=ws)
    assert out[0] is buf and out[1] is h and torch.equal(buf, y) and torch.equal(h, hl)
    out = bd.ssm_gated_scan_fwd(**d, want_h_last=False)
    assert out[1] is None and torch.equal(out[0], y)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh)
    dx = torch.empty_like(y)
    k = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, want_dh0=False, want_dlog_a=False, grads={"dx": dx})
    assert set(k) == {"dx", "dga", "dgx", "dz"} and k["dx"] is dx
    for n in k:
        assert torch.equal(k[n], g[n]), n
    with pytest.raises(ValueError, match="unknown output"):
        bd.ssm_gated_scan_bwd(**d, dy=dy, grads={"dq": dx})
    with pytest.raises(bd.SsmError):
        bd.ssm_gated_scan_fwd(**d, y=d["x"])


@pytest.mark.parametrize("B,L,D", [(0, 5, 8), (2, 0, 8), (2, 5, 0)])
def test_empty(lib, B, L, D):
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(9, B, L, D, "f32", fused=False)
    y, hl, ck = bd.ssm_gated_scan_fwd(**d, want_ckpt=True)
    assert y.shape == (B, L, D) and torch.equal(hl, d["h0"])
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck)
    assert g["dx"].shape == (B, L, D) and torch.equal(g["dh0"], dh) and not g["dlog_a"].any()


@pytest.mark.parametrize("L,cut", [(300, 77), (1500, 640), (1100, 1)])
def test_resume(lib, L, cut):
    """A sequence in two calls: the second continues the first's state (fp32: within the bounds of both)."""
    from selective_state_space_84_amd import binding as bd
    d, _, _ = _make(10, 1, L, 66, "f32")
    ref = P.scan(**{k: _np(v) for k, v in d.items()})
    part = lambda a, b, h: bd.ssm_gated_scan_fwd(  # noqa: E731
        **{k: v[:, a:b] for k, v in d.items() if k in ("x", "ga", "gx", "z")}, log_a=d["log_a"], h0=h)
    y1, h1, _ = part(0, cut, d["h0"])
    y2, h2, _ = part(cut, L, h1)
    tol = P.tol(*ref["y"], "f32")
    _close("y1", _np(y1), ref["y"][0][:, :cut], tol[:, :cut])
    _close("y2", _np(y2), ref["y"][0][:, cut:], tol[:, cut:])
    _close("h", _np(h2), ref["h_last"][0], P.tol(*ref["h_last"], "f32"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("B,D,pad", [(1, 1, 2), (1, 2048, 4), (3, 70, 2), (7, 333, 3), (64, 520, 4), (5, 260, 1),
                                     (9, 1028, 8), (2, 4, 4)])
def test_update(lib, B, D, pad, z, dtype):
    """Rows read in fours (widths and distances that are multiples of four) and one by one."""
    import torch
    from selective_state_space_84_amd import binding as bd
    print("case", B, D, pad, z, dtype, flush=True)
    d, _, _ = _make(B + D, B, 1, D, dtype, z=z, pad=pad)
    d = {k: v[:, 0] if k in ("x", "ga", "gx", "z") and v is not None else v for k, v in d.items()}
    slots = None
    if B > 1:
        slots = [(2 * i + 1) % (2 * B) if i % 5 != 3 else (-1 if i % 2 else 2 * B + 7) for i in range(B)]
    h = _t(np.random.default_rng(B).standard_normal((B if slots is None else 2 * B + 1, D)))
    ins = {k: _np(v) for k, v in d.items() if k != "h0"}
    (y, hn) = P.update(_np(h), **ins, slots=slots)
    d.pop("h0")
    got = bd.ssm_gated_scan_update(h, **d, slots=_lens(slots))
    torch.cuda.synchronize()
    _close("y", _np(got), y[0], P.tol(*y, dtype))
    _close("h", _np(h), hn[0], P.tol(*hn, "f32"))
    for b, k in enumerate(slots or []):
        assert 0 <= k < h.shape[0] or not got[b].any()


def test_update_large_offsets(lib):
    """A cache beyond 2^31 elements, and rows whose distance passes 2^31 bytes."""
    import torch
    from selective_state_space_84_amd import binding as bd
    D, n = 8192, 270000
    h = torch.empty(n, D, device=DEV)
    d, _, _ = _make(11, 2, 1, D, "bf16", fused=False)
    far = torch.empty(2, 1 << 17, D, dtype=torch.bfloat16, device=DEV)
    far[:, 0] = d["ga"][:, 0]
    slots = [n - 1, 1]
    h[[n - 1, 1]] = d["h0"]
    h[n - 2] = 5.0
    args = dict(x=d["x"][:, 0], ga=far[:, 0], gx=d["gx"][:, 0], log_a=d["log_a"], z=d["z"][:, 0])
    y, hn = P.update(_np(d["h0"]), **{k: _np(v) for k, v in args.items()}, slots=[0, 1])
    got = bd.ssm_gated_scan_update(h, **args, slots=_lens(slots))
    _close("y", _np(got), y[0], P.tol(*y, "bf16"))
    _close("h", _np(h[[n - 1, 1]]), hn[0], P.tol(*hn, "f32"))
    assert (h[n - 2] == 5.0).all()


def test_scan_large_offsets(lib):
    """Inputs and outputs of more than 2^31 elements: the last channels against the same ones alone."""
    import torch
    from selective_state_space_84_amd import binding as bd
    B, L, D = 2, 140000, 8192
    x = torch.empty(B, L, D, dtype=torch.bfloat16, device=DEV).normal_()
    log_a = -torch.rand(D, device=DEV)
    y, hl, ck = bd.ssm_gated_scan_fwd(x, x, x, log_a, want_ckpt=True)
    cut = x[:, :, D - 64:].contiguous()
    y1, h1, _ = bd.ssm_gated_scan_fwd(cut, cut, cut, log_a[D - 64:].contiguous())
    assert torch.equal(y[:, :, D - 64:], y1) and torch.equal(hl[:, D - 64:], h1)
    g = bd.ssm_gated_scan_bwd(x, x, x, log_a, dy=y, ckpt=ck)
    g1 = bd.ssm_gated_scan_bwd(cut, cut, cut, log_a[D - 64:].contiguous(), dy=y1)
    for n in ("dx", "dga", "dgx"):
        assert torch.equal(g[n][:, :, D - 64:], g1[n]), n
    assert torch.equal(g["dh0"][:, D - 64:], g1["dh0"])


def test_more_pieces_than_a_launch(lib):
    """1.5 million rows of three pieces (gradient: five) take several launches: sampled rows against the same alone."""
    import torch
    from selective_state_space_84_amd import binding as bd
    B, L = 1500000, 300
    x = torch.empty(B, L, 1, dtype=torch.bfloat16, device=DEV).normal_()
    log_a = torch.tensor([-0.05], device=DEV)
    lens = torch.randint(0, L + 1, (B,), dtype=torch.int32, device=DEV)
    y, hl, ck = bd.ssm_gated_scan_fwd(x, x, x, log_a, lengths=lens, want_ckpt=True)
    g = bd.ssm_gated_scan_bwd(x, x, x, log_a, dy=x, lengths=lens, ckpt=ck, want_dlog_a=False)
    for r in (0, 699050, 1048575, 1398102, B - 3):  # around the launches' borders
        cut, n = x[r:r + 3].clone(), lens[r:r + 3].clone()
        y1, h1, _ = bd.ssm_gated_scan_fwd(cut, cut, cut, log_a, lengths=n)
        g1 = bd.ssm_gated_scan_bwd(cut, cut, cut, log_a, dy=cut, lengths=n, want_dlog_a=False)
        assert torch.equal(y[r:r + 3], y1) and torch.equal(hl[r:r + 3], h1), r
        for k in g1:
            assert torch.equal(g[k][r:r + 3], g1[k]), (r, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_widest_rows_and_strides(lib, dtype):
    """The largest width, and the largest distance between steps."""
    import torch
    from selective_state_space_84_amd import binding as bd
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    D = 1 << 23
    x = torch.empty(1, 3, D, dtype=dt, device=DEV).normal_()
    log_a = -torch.rand(D, device=DEV)
    y, hl, _ = bd.ssm_gated_scan_fwd(x, x, x, log_a)
    g = bd.ssm_gated_scan_bwd(x, x, x, log_a, dy=y)
    cut, la = x[:, :, D - 130:].contiguous(), log_a[D - 130:].contiguous()
    y1, h1, _ = bd.ssm_gated_scan_fwd(cut, cut, cut, la)
    g1 = bd.ssm_gated_scan_bwd(cut, cut, cut, la, dy=y1)
    assert torch.equal(y[:, :, D - 130:], y1) and torch.equal(hl[:, D - 130:], h1)
    for k in g1:
        assert torch.equal(g[k][..., D - 130:], g1[k]), k
    del x, y, g
    far = torch.empty(1, 18, 1 << 25, dtype=dt, device=DEV)
    far[:, :, 64:194].normal_()
    v = far[:, :, 64:194]
    y, hl, _ = bd.ssm_gated_scan_fwd(v, v, v, la)
    c = v.contiguous()
    y1, h1, _ = bd.ssm_gated_scan_fwd(c, c, c, la)
    assert torch.equal(y, y1) and torch.equal(hl, h1)
    a, b = bd.ssm_gated_scan_bwd(v, v, v, la, dy=y), bd.ssm_gated_scan_bwd(c, c, c, la, dy=y)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_zeros_behind_a_row_whatever_comes_from_there(lib):
    """A gradient of the last state that is not finite reaches the row's steps and nothing behind them."""
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(18, 3, 200, 70, "bf16")
    dh[:] = float("inf")
    dh[1] = float("nan")
    lens = [150, 64, 0]
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, lengths=_lens(lens))
    for b, n in enumerate(lens):
        for k in ("dx", "dga", "dgx", "dz"):
            assert not g[k][b, n:].any(), (b, k)
    assert torch.isnan(g["dx"][1, :64]).all() and torch.equal(g["dh0"][2], dh[2])


def test_prompt_then_tokens(lib):
    """A prompt continued token by token equals one longer prompt, through the norms around it."""
    import torch
    from selective_state_space_84_amd import binding as bd
    B, L, D, n = 3, 200, 128, 5
    d, _, _ = _make(12, B, L + n, D, "f32", states=False)
    lens = torch.tensor([L, 100, L - 7], dtype=torch.int32, device=DEV)
    full = bd.ssm_gated_scan_fwd(**d)[0]
    keys = ("x", "ga", "gx", "z")
    _, h, _ = bd.ssm_gated_scan_fwd(**{**d, **{k: d[k][:, :L].contiguous() for k in keys}}, lengths=lens)
    cache = torch.zeros(7, D, device=DEV)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device=DEV)
    cache[slots.long()] = h
    for i in range(n):
        at = [int(v) + i for v in lens]
        tok = {k: torch.stack([d[k][b, t] for b, t in enumerate(at)]) for k in keys}
        y = bd.ssm_gated_scan_update(cache, **tok, log_a=d["log_a"], slots=slots)
        want = torch.stack([full[b, t] for b, t in enumerate(at)])
        assert torch.allclose(y, want, rtol=2e-5, atol=2e-5)


def test_other_stream_and_device_order(lib):
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(13, 2, 900, 130, "bf16")
    want = bd.ssm_gated_scan_fwd(**d, want_ckpt=True)
    wg = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=want[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = bd.ssm_gated_scan_fwd(**d, want_ckpt=True, stream=s)
    g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=got[2], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n in g:
        assert torch.equal(g[n], wg[n]), n


def test_graph_capture(lib):
    """A training step captured once: every replay equals the eager call, with eager work between."""
    import torch
    from selective_state_space_84_amd import binding as bd
    d, dy, dh = _make(14, 2, 1000, 130, "bf16")

    def step():
        y, hl, ck = bd.ssm_gated_scan_fwd(**d, want_ckpt=True)
        g = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck)
        k = bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh)
        return [y, hl, *g.values(), *k.values()]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        d["x"].mul_(1.25)
        dy.mul_(0.75)
        want = step()
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), i


def test_two_at_once(lib):
    """Calls on two streams at the same time, each with its own workspace, bitwise as alone."""
    import torch
    from selective_state_space_84_amd import binding as bd
    a, b = _make(15, 4, 4096, 512, "bf16"), _make(16, 4, 4096, 512, "bf16")

    def step(m, stream=None):
        d, dy, dh = m
        y, hl, ck = bd.ssm_gated_scan_fwd(**d, want_ckpt=True, stream=stream)
        return [y, hl, *bd.ssm_gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck, stream=stream).values()]
    want = [step(a), step(b)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = [step(a, streams[0]), step(b, streams[1])]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, g))


def test_training_step_against_differences(lib):
    """Norm, gated recurrence, gated norm and residual norm together, as a layer runs them: gradients against
    differences of the loss (fp32)."""
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(17)
    B, L, D = 2, 150, 64
    p = {n: _t(r.standard_normal((B, L, D))) for n in ("x", "res", "ga", "gx", "z")}
    w = {n: _t(1 + 0.2 * r.standard_normal(D)) for n in ("w0", "w1", "w2", "w3")}
    log_a = _t(-np.exp(r.uniform(-4, 1, D)))
    dy, dR = _t(r.standard_normal((B, L, D))), _t(r.standard_normal((B, L, D)))

    def forward():
        r1, n1 = bd.ssm_residual_norm_fwd(p["x"], p["res"], w["w0"])
        y, _, ck = bd.ssm_gated_scan_fwd(n1, p["ga"], p["gx"], log_a, want_ckpt=True)
        o = bd.ssm_gated_norm_fwd(y, p["z"], w["w1"], groups=2)
        r2, n2 = bd.ssm_residual_norm_fwd(o, r1, w["w2"], w["w3"], alpha=0.5, post_norm=True)
        return r1, n1, y, ck, o, r2, n2

    def loss():
        out = forward()
        return float((out[6].double() * dy.double()).sum() + (out[5].double() * dR.double()).sum())
    r1, n1, y, ck, o, r2, n2 = forward()
    g2 = bd.ssm_residual_norm_bwd(o, r2, w["w2"], w["w3"], dy=dy, dres_out=dR, alpha=0.5, post_norm=True)
    gn = bd.ssm_gated_norm_bwd(y, p["z"], w["w1"], dy=g2["dx"], groups=2)
    gs = bd.ssm_gated_scan_bwd(n1, p["ga"], p["gx"], log_a, dy=gn["dx"], ckpt=ck, want_dh0=False)
    g1 = bd.ssm_residual_norm_bwd(p["x"], r1, w["w0"], dy=gs["dx"], dres_out=g2["dres"])
    grads = {"x": g1["dx"], "res": g1["dres"], "ga": gs["dga"], "gx": gs["dgx"], "z": gn["dz"], "log_a": gs["dlog_a"],
             "w0": g1["dw_pre"], "w1": gn["dw"], "w2": g2["dw_pre"], "w3": g2["dw_post"]}
    leaves = {**p, **w, "log_a": log_a}
    for n, g in grads.items():
        v = _t(r.standard_normal(g.shape)) * (leaves[n].abs().mean() if n == "log_a" else 1.0)
        if n == "log_a":
            v = v * leaves[n].abs()
        h = 1e-2
        old = leaves[n].clone()
        leaves[n].copy_(old + h * v)
        up = loss()
        leaves[n].copy_(old - h * v)
        down = loss()
        leaves[n].copy_(old)
        num, ana = (up - down) / (2 * h), float((g.double() * v.double()).sum())
        # The loss sums 4 * 10^4 terms of size 1 with errors of 1e-6: +-2e-4 random, over 2 h 1e-2; the third derivative
        # times h^2 / 6 is 1.7e-5 of a few hundred.
        scale = float(g.double().norm() * v.double().norm())
        assert abs(num - ana) <= 2e-2 + 1e-3 * scale, (n, num, ana, scale)
