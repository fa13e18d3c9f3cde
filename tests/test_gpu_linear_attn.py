"""Linear attention with a decay per head (whole sequences, gradient, one step)
against the 64-bit definitions, elementwise within the bounds of plain64.py."""
import numpy as np
import pytest

import plain64 as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _t(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.as_tensor(np.ascontiguousarray(a), dtype=torch.float32)
    return (t.to(torch.bfloat16) if dtype == "bf16" else t).to(DEV)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _make(seed, B, L, H, M, K, V, dtype, states=True, fused=False, decay=None):
    """Inputs on the device, and the same values in 64 bits."""
    import torch
    r = np.random.default_rng(seed)
    if fused:  # column ranges of one projection's output, with unused columns between
        W = H * K + M * (K + V) + 32
        wide = _t(r.standard_normal((B, L, W)), dtype)
        q = wide[:, :, :H * K].unflatten(2, (H, K))
        k = wide[:, :, H * K + 16:H * K + 16 + M * K].unflatten(2, (M, K))
        v = wide[:, :, W - M * V:].unflatten(2, (M, V))
    else:
        q, k, v = (_t(r.standard_normal((B, L, h, d)), dtype) for h, d in ((H, K), (M, K), (M, V)))
    if decay is None:
        decay = -np.exp(r.uniform(-6, 0, H))
    g = _t(np.asarray(decay, dtype=np.float32))
    h0 = _t(r.standard_normal((B, H, V, K))) if states else None
    d = dict(q=q, k=k, v=v, log_decay=g, h0=h0)
    do, dh = _t(r.standard_normal((B, L, H, V)), dtype), (_t(r.standard_normal((B, H, V, K))) if states else None)
    torch.cuda.synchronize()
    return d, {n: _np(t) for n, t in d.items()}, do, dh


def _close(name, got, ref, tol):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    print("  %s: worst error / bound %.3f" % (name, worst), flush=True)
    assert not bad.any(), "%s: %d of %d out of bounds, worst %.3g" % (name, bad.sum(), bad.size, worst)


def _check_fwd(d, n, dtype, lengths=None, scale=None, **kw):
    import torch
    from selective_state_space_84_amd import binding
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    o, hl = binding.ssm_linear_attn_fwd(**d, lengths=lens, scale=scale, **kw)
    torch.cuda.synchronize()
    ro, rh = P.attn_fwd(**n, lengths=lengths, scale=scale)
    mo, mh = P.attn_fwd_mag(**n, lengths=lengths, scale=scale)
    L, K = n["q"].shape[1], n["q"].shape[3]
    _close("o", _np(o), ro, P.attn_tol(ro, mo, L, K, dtype))
    _close("h_last", _np(hl), rh, P.attn_tol(rh, mh, L, K, "f32"))
    return o, hl


def _check_bwd(d, n, do, dh, dtype, lengths=None, scale=None, **kw):
    import torch
    from selective_state_space_84_amd import binding
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    g = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh, lengths=lens, scale=scale, **kw)
    torch.cuda.synchronize()
    args = dict(n, do=_np(do), dh_last=_np(dh), lengths=lengths, scale=scale)
    ref, mag = P.attn_bwd(**args), P.attn_bwd_mag(**args)
    L, W = n["q"].shape[1], max(n["q"].shape[3], n["v"].shape[3])
    rep = n["q"].shape[2] // n["k"].shape[2]
    for name, r, m in zip(("dq", "dk", "dv", "dh0"), ref, mag):
        _close(name, _np(g[name]), r, P.attn_tol(r, m, L, W, "f32" if name == "dh0" else dtype, rep))
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 300])
def test_lengths(lib, L, dtype):
    print("case", L, dtype, flush=True)
    d, n, do, dh = _make(L, 2, L, 2, 1, 64, 128, dtype)
    _check_fwd(d, n, dtype)
    _check_bwd(d, n, do, dh, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,M", [(1, 1), (6, 3), (4, 1)])
def test_widths_heads_and_strides(lib, K, V, H, M, dtype):
    print("case", K, V, H, M, dtype, flush=True)
    d, n, do, dh = _make(K + V + H, 2, 77, H, M, K, V, dtype, fused=True)
    _check_fwd(d, n, dtype)
    _check_bwd(d, n, do, dh, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("states", [False, True])
def test_padded_batch(lib, states, dtype):
    """Rows of 0, 1, some and all steps (and lengths outside the range, which are
    clamped); what lies behind a row's length is NaN and must not be used."""
    import torch
    lengths = [300, 0, 1, 129, 64, 500, -3]
    d, n, do, dh = _make(7, len(lengths), 300, 2, 2, 64, 64, dtype, states=states)
    for b, l in enumerate(lengths):
        for t in (d["q"], d["k"], d["v"], do):
            t[b, max(l, 0):] = float("nan")
    n = {k: np.nan_to_num(v) if v is not None else None for k, v in ((k, _np(t)) for k, t in d.items())}
    o, hl = _check_fwd(d, n, dtype, lengths)
    assert not o[1].any() and not o[6].any()
    if states:
        assert torch.equal(hl[1], d["h0"][1])
    from selective_state_space_84_amd import binding
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    g = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh, lengths=lens)
    torch.cuda.synchronize()
    args = dict(n, do=np.nan_to_num(_np(do)), dh_last=_np(dh), lengths=lengths)
    for name, r, m in zip(("dq", "dk", "dv", "dh0"), P.attn_bwd(**args), P.attn_bwd_mag(**args)):
        _close(name, _np(g[name]), r, P.attn_tol(r, m, 300, 64, "f32" if name == "dh0" else dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_extremes(lib, dtype):
    """No decay, total decay, decays whose powers leave fp32's range within a block, and hardly any."""
    dec = [0.0, -np.inf, -80.0, -3.0, -1e-7]
    d, n, do, dh = _make(8, 1, 200, 5, 5, 64, 64, dtype, decay=dec)
    _check_fwd(d, n, dtype)
    _check_bwd(d, n, do, dh, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_spans(lib, dtype):
    """Few heads and a long sequence: cut into spans, entry states carried between them, rows ending inside one."""
    from selective_state_space_84_amd import binding
    B, L = 2, 1100
    assert binding.load_library().ssm_linear_attn_fwd_workspace_size(B, L, 1, 64, 128, 1 if dtype == "bf16" else 0) > 0
    d, n, do, dh = _make(9, B, L, 1, 1, 64, 128, dtype, decay=[-1e-3])
    _check_fwd(d, n, dtype, [1100, 413])
    _check_bwd(d, n, do, dh, dtype, [1100, 413])


def test_options(lib):
    """scale, absent states, no h_last, no dh0; and no NaN from unwritten memory: outputs given, filled with NaN."""
    import torch
    from selective_state_space_84_amd import binding
    d, n, do, dh = _make(10, 2, 50, 2, 2, 64, 64, "bf16", states=False)
    o = torch.full((2, 50, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    got, hl = binding.ssm_linear_attn_fwd(**d, scale=-2.5, o=o, want_h_last=False)
    assert got is o and hl is None
    ro, _ = P.attn_fwd(**n, scale=-2.5)
    mo, _ = P.attn_fwd_mag(**n, scale=-2.5)
    _close("o", _np(o), ro, P.attn_tol(ro, mo, 50, 64, "bf16"))
    grads = {k: torch.full(tuple(d[k[1]].shape), float("nan"), dtype=torch.bfloat16, device=DEV)
             for k in ("dq", "dk", "dv")}
    g = binding.ssm_linear_attn_bwd(**d, do=do, scale=-2.5, want_dh0=False, grads=grads)
    assert set(g) == {"dq", "dk", "dv"} and g["dq"] is grads["dq"]
    args = dict(n, do=_np(do), scale=-2.5)
    for name, r, m in zip(("dq", "dk", "dv"), P.attn_bwd(**args), P.attn_bwd_mag(**args)):
        _close(name, _np(g[name]), r, P.attn_tol(r, m, 50, 64, "bf16"))


def test_empty_sequence(lib):
    import torch
    from selective_state_space_84_amd import binding
    d, _, do, dh = _make(11, 2, 0, 2, 2, 64, 128, "bf16")
    o, hl = binding.ssm_linear_attn_fwd(**d)
    assert o.shape == (2, 0, 2, 128) and torch.equal(hl, d["h0"])
    g = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh)
    assert torch.equal(g["dh0"], dh) and g["dq"].numel() == 0


@pytest.mark.parametrize("L,cut", [(300, 77), (1500, 640)])
def test_resume_in_place_and_repeat(lib, L, cut):
    """A sequence in two calls, the state handed over in one buffer, equals one call; calls repeat bitwise."""
    import torch
    from selective_state_space_84_amd import binding
    d, n, _, _ = _make(12, 1, L, 2, 2, 64, 64, "f32")
    o, hl = binding.ssm_linear_attn_fwd(**d)
    o2, hl2 = binding.ssm_linear_attn_fwd(**d)
    assert torch.equal(o, o2) and torch.equal(hl, hl2)
    st = d["h0"].clone()
    parts = []
    for sl in (slice(0, cut), slice(cut, L)):
        a, b = binding.ssm_linear_attn_fwd(d["q"][:, sl], d["k"][:, sl], d["v"][:, sl], d["log_decay"], h0=st, h_last=st)
        assert b is st
        parts.append(a)
    mo, mh = P.attn_fwd_mag(**n)
    # Both sides are within the bound of the definition.
    _close("o", _np(torch.cat(parts, 1)), _np(o), 2 * P.attn_tol(_np(o), mo, L, 64, "f32"))
    _close("h_last", _np(st), _np(hl), 2 * P.attn_tol(_np(hl), mh, L, 64, "f32"))


# ---- one step --------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H,M", [(1, 1, 1), (3, 6, 2), (40, 16, 16)])
def test_update(lib, B, H, M, K, V, dtype):
    import torch
    from selective_state_space_84_amd import binding
    d, n, _, _ = _make(B + K + V, B, 1, H, M, K, V, dtype, fused=True)
    h = d["h0"].clone()
    o = binding.ssm_linear_attn_update(h, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"])
    torch.cuda.synchronize()
    ro, rh = P.attn_fwd(**n)
    mo, mh = P.attn_fwd_mag(**n)
    _close("o", _np(o), ro[:, 0], P.attn_tol(ro, mo, 1, K, dtype)[:, 0])
    _close("h", _np(h), rh, P.attn_tol(rh, mh, 1, 0, "f32"))


def test_update_slots(lib):
    """States anywhere in a cache; unused rows (negative or beyond the cache) touch nothing and give zeros."""
    import torch
    from selective_state_space_84_amd import binding
    slots = [5, -1, 0, 9, 3, 1 << 30, -(1 << 31), 8]
    B, n_slots = len(slots), 9
    used = [i for i, s in enumerate(slots) if 0 <= s < n_slots]
    d, n, _, _ = _make(13, B, 1, 4, 2, 64, 128, "bf16")
    cache = torch.randn(n_slots, 4, 128, 64, device=DEV)
    for i in used:
        cache[slots[i]] = d["h0"][i]
    before = cache.clone()
    o = torch.full((B, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    binding.ssm_linear_attn_update(cache, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], o=o,
                                   slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ro, rh = P.attn_fwd(**n)
    mo, mh = P.attn_fwd_mag(**n)
    for i, s in enumerate(slots):
        if i in used:
            _close("o", _np(o[i]), ro[i, 0], P.attn_tol(ro, mo, 1, 64, "bf16")[i, 0])
            _close("h", _np(cache[s]), rh[i], P.attn_tol(rh, mh, 1, 0, "f32")[i])
        else:
            assert not o[i].any()
    for s in set(range(n_slots)) - {slots[i] for i in used}:
        assert torch.equal(cache[s], before[s])


def test_update_large_offsets(lib):
    """A cache of more than 2^31 elements: states beyond 32-bit byte and element offsets."""
    import torch
    from selective_state_space_84_amd import binding
    n_slots = (1 << 31) // (32 * 128 * 128) + 3  # 2^31 elements and a little more, 8.6 GB
    cache = torch.empty(n_slots, 32, 128, 128, device=DEV)
    slots = [n_slots - 1, 1, n_slots // 2 + 1]
    d, n, _, _ = _make(14, 3, 1, 32, 32, 128, 128, "bf16")
    for i, s in enumerate(slots):
        cache[s] = d["h0"][i]
    o = binding.ssm_linear_attn_update(cache, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"],
                                       slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ro, rh = P.attn_fwd(**n)
    mo, mh = P.attn_fwd_mag(**n)
    _close("o", _np(o), ro[:, 0], P.attn_tol(ro, mo, 1, 128, "bf16")[:, 0])
    for i, s in enumerate(slots):
        _close("h", _np(cache[s]), rh[i], P.attn_tol(rh, mh, 1, 0, "f32")[i])


# ---- together, streams, graphs ---------------------------------------------

def test_prompt_then_tokens(lib):
    """Norm and rotation, a prompt, then tokens through the one-step form from a
    slot cache: the last outputs equal those of the whole sequence in one call."""
    import torch
    from selective_state_space_84_amd import binding
    B, L, T, H, M, K, V = 2, 70, 6, 4, 2, 64, 64
    r = np.random.default_rng(15)
    wide = _t(r.standard_normal((B, L + T, H * K + M * (K + V))), "f32")
    w = _t(1 + 0.1 * r.standard_normal(K))
    f = _t(10000.0 ** (-np.arange(16) / 16.0))
    g = _t([-0.01, -0.1, 0.0, -1.0])

    def layer(x, pos):
        q = x[:, :, :H * K].unflatten(2, (H, K))
        k = x[:, :, H * K:(H + M) * K].unflatten(2, (M, K))
        v = x[:, :, (H + M) * K:].unflatten(2, (M, V))
        q, k = binding.ssm_qk_norm_rope_fwd(q, k, w, w, f, positions=pos)
        return q, k, v
    pos = torch.arange(1000, 1000 + L + T, device=DEV).repeat(B, 1)
    q, k, v = layer(wide, pos)
    whole, last = binding.ssm_linear_attn_fwd(q, k, v, g)
    q0, k0, v0 = layer(wide[:, :L].contiguous(), pos[:, :L].contiguous())
    _, st = binding.ssm_linear_attn_fwd(q0, k0, v0, g)
    cache = torch.zeros(5, H, V, K, device=DEV)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    cache[slots.long()] = st
    n = dict(q=_np(q), k=_np(k), v=_np(v), log_decay=_np(g))
    mo, mh = P.attn_fwd_mag(**n)
    for t in range(L, L + T):
        q1, k1, v1 = layer(wide[:, t:t + 1].contiguous(), pos[:, t:t + 1].contiguous())
        o = binding.ssm_linear_attn_update(cache, q1[:, 0], k1[:, 0], v1[:, 0], g, slots=slots)
        _close("o", _np(o), _np(whole[:, t]), 2 * P.attn_tol(_np(whole), mo, L + T, K, "f32")[:, t])
    _close("state", _np(cache[slots.long()]), _np(last), 2 * P.attn_tol(_np(last), mh, L + T, K, "f32"))


def test_training_step_against_differences(lib):
    """Norm, rotation and attention with their gradients chained: the derivative
    of a loss along random directions of q, k and v, against central differences."""
    import torch
    from selective_state_space_84_amd import binding
    B, L, H, M, K, V = 1, 40, 2, 1, 64, 64
    r = np.random.default_rng(16)
    q, k, v = (_t(r.standard_normal((B, L, h, d))) for h, d in ((H, K), (M, K), (M, V)))
    wq, wk, f, g = _t(np.ones(K)), _t(np.ones(K)), _t(r.random(32)), _t([-0.05, -0.5])
    do = _t(r.standard_normal((B, L, H, V)))
    qn, kn = binding.ssm_qk_norm_rope_fwd(q, k, wq, wk, f)
    a = binding.ssm_linear_attn_bwd(qn, kn, v, g, do=do)
    n = binding.ssm_qk_norm_rope_bwd(q, k, wq, wk, f, dq_out=a["dq"], dk_out=a["dk"])
    pos = np.arange(L)[None].repeat(B, 0)

    def loss(q, k, v, wq, wk):
        qn = P.norm_rope(q, wq, pos, _np(f), 1e-6, False)[0]
        kn = P.norm_rope(k, wk, pos, _np(f), 1e-6, False)[0]
        return (P.attn_fwd(qn, kn, v, _np(g))[0] * _np(do)).sum()
    x = [_np(t) for t in (q, k, v, wq, wk)]
    grads = [_np(t) for t in (n["dq"], n["dk"], a["dv"], n["dwq"], n["dwk"])]
    for i, gr in enumerate(grads):
        dirn = r.standard_normal(x[i].shape)
        e = 1e-5
        up = loss(*[t + e * dirn if j == i else t for j, t in enumerate(x)])
        dn = loss(*[t - e * dirn if j == i else t for j, t in enumerate(x)])
        num, ana = (up - dn) / (2 * e), float((gr * dirn).sum())
        # fp32 gradients: 2^-17 of the sum of their absolute shares covers some hundred roundings each.
        bound = 2.0 ** -17 * np.abs(gr * dirn).sum() + 1e-6 * abs(num)
        print("  direction %d: %.8g %.8g" % (i, num, ana), flush=True)
        assert abs(num - ana) <= bound


def test_other_stream(lib):
    """Calls on a stream of their own, workspaces and outputs included, while the current one works on."""
    import torch
    from selective_state_space_84_amd import binding
    d, n, do, dh = _make(17, 1, 1200, 2, 1, 64, 64, "bf16")
    want = binding.ssm_linear_attn_fwd(**d)
    wg = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = binding.ssm_linear_attn_fwd(**d, stream=s)
        g = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh, stream=s.cuda_stream)
        torch.randn(1 << 20, device=DEV).sum()
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for name in wg:
            assert torch.equal(g[name], wg[name]), name


def test_graph_capture(lib):
    """Prompt, gradient and one step captured in a graph; every replay equals the eager calls."""
    import torch
    from selective_state_space_84_amd import binding
    d, n, do, dh = _make(18, 1, 700, 2, 1, 64, 64, "bf16")
    h = d["h0"].clone()

    def step():
        o, hl = binding.ssm_linear_attn_fwd(**d)
        g = binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh)
        u = binding.ssm_linear_attn_update(h, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"])
        return [o, hl, g["dq"], g["dk"], g["dv"], g["dh0"], u]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    r = np.random.default_rng(19)
    for _ in range(3):
        for name in ("q", "k", "v"):
            d[name].copy_(_t(r.standard_normal(tuple(d[name].shape)), "bf16"))
        keep = h.clone()
        want = [t.clone() for t in step()]
        hw = h.clone()
        h.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(h, hw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,M", [(70000, 1, 1), (1, 32768, 8)])
def test_many_rows_and_heads(lib, B, H, M, dtype):
    """More rows than a 16-bit grid axis, and the most heads: prompt of two steps, gradient of v, one token."""
    import torch
    from selective_state_space_84_amd import binding
    print("case", B, H, M, dtype, flush=True)
    r = np.random.default_rng(21)
    q, k, v = (_t(r.standard_normal((B, 2, h, 64)), dtype) for h in (H, M, M))
    dec = _t(-r.random(H))
    rep = H // M
    nq, nk, nv = _np(q), np.repeat(_np(k), rep, 2), np.repeat(_np(v), rep, 2)
    g = np.exp(_np(dec))[None, :, None]

    def pairs(f):  # scale * (q_1 . k_i), i = 0 (decayed) and 1, with f applied to the factors
        return [64 ** -0.5 * (f(nq[:, 1]) * f(nk[:, i])).sum(-1, keepdims=True) * (g if i == 0 else 1) for i in (0, 1)]
    a, m = pairs(lambda x: x), pairs(np.abs)
    ref, mag = (p[0] * f(nv[:, 0]) + p[1] * f(nv[:, 1]) for p, f in ((a, lambda x: x), (m, np.abs)))
    o, none = binding.ssm_linear_attn_fwd(q, k, v, dec, want_h_last=False)
    assert none is None
    _close("o", _np(o[:, 1]), ref, P.attn_tol(ref, mag, 2, 64, dtype))
    # dv of the last step is its own pair's weight times do, summed over the heads that share v.
    do = torch.zeros_like(o)
    do[:, 1] = 1
    gr = binding.ssm_linear_attn_bwd(q, k, v, dec, do=do, want_dh0=False)
    dv, dm = (p[1].reshape(B, M, rep, 1).sum(2) * np.ones(64) for p in (a, m))
    _close("dv", _np(gr["dv"][:, 1]), dv, P.attn_tol(dv, dm, 2, 64, dtype, rep))
    h = torch.zeros(B, H, 64, 64, device=DEV)
    binding.ssm_linear_attn_update(h, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), dec)
    u = binding.ssm_linear_attn_update(h, q[:, 1].contiguous(), k[:, 1].contiguous(), v[:, 1].contiguous(), dec)
    _close("u", _np(u), ref, P.attn_tol(ref, mag, 2, 64, dtype))


def test_two_at_once(lib):
    """Calls in flight on two streams, each with its own workspace, and outputs given by the caller."""
    import torch
    from selective_state_space_84_amd import binding
    sets = [_make(22 + i, 1, 2500, 2, 1, 128, 128, "bf16") for i in range(2)]
    want = []
    for d, _, do, dh in sets:
        want.append((binding.ssm_linear_attn_fwd(**d), binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    given = [torch.empty_like(d["q"], memory_format=torch.contiguous_format) for d, _, _, _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (d, _, do, dh) in enumerate(sets):
            got[i].append((binding.ssm_linear_attn_fwd(**d, stream=streams[i]),
                           binding.ssm_linear_attn_bwd(**d, do=do, dh_last=dh, stream=streams[i],
                                                       grads={"dq": given[i]})))
    torch.cuda.synchronize()
    for i in range(2):
        for f, g in got[i]:
            assert g["dq"] is given[i]
            assert torch.equal(f[0], want[i][0][0]) and torch.equal(f[1], want[i][0][1])
            assert all(torch.equal(g[name], want[i][1][name]) for name in g)
    # 0 is the default stream's handle.
    d = sets[0][0]
    o, _ = binding.ssm_linear_attn_fwd(**d, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0][0])
