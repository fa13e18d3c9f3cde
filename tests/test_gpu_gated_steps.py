"""A training step through the residual norms, the gated recurrence and the gated
norm: each leaf's gradient against differences of the loss along the signs of that
gradient, so that an error in proportion to it shows whatever the leaf's size
(fp32)."""
import numpy as np
import pytest

from test_gpu_linear_attn import _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,gate_first,post", [(2, True, True), (1, False, False)])
def test_gradients_along_their_signs(lib, groups, gate_first, post):
    import torch
    from selective_state_space_84_amd import binding as bd
    r = np.random.default_rng(3)
    B, L, D = 2, 150, 64
    p = {n: _t(r.standard_normal((B, L, D))) for n in ("x", "res", "ga", "gx", "z")}
    w = {n: _t(1 + 0.2 * r.standard_normal(D)) for n in ("w0", "w1", "w2", "w3")}
    log_a, h0 = _t(-np.exp(r.uniform(-4, 1, D))), _t(r.standard_normal((B, D)))
    dy, dR, dh = (_t(r.standard_normal(s)) for s in ((B, L, D), (B, L, D), (B, D)))
    lens = torch.tensor([L, 77], dtype=torch.int32, device=dy.device)

    def forward():
        r1, n1 = bd.ssm_residual_norm_fwd(p["x"], p["res"], w["w0"])
        y, hl, ck = bd.ssm_gated_scan_fwd(n1, p["ga"], p["gx"], log_a, p["z"], lengths=lens, h0=h0, want_ckpt=True)
        o = bd.ssm_gated_norm_fwd(y, p["gx"], w["w1"], groups=groups, gate_first=gate_first, eps=1e-2)
        r2, n2 = bd.ssm_residual_norm_fwd(o, r1, w["w2"], w["w3"], alpha=0.5, post_norm=post, eps=1e-2)
        return r1, n1, y, ck, o, r2, n2, hl

    def loss():
        out = forward()
        return float((out[6].double() * dy.double()).sum() + (out[5].double() * dR.double()).sum() +
                     (out[7].double() * dh.double()).sum())
    r1, n1, y, ck, o, r2, n2, hl = forward()
    g2 = bd.ssm_residual_norm_bwd(o, r2, w["w2"], w["w3"], dy=dy, dres_out=dR, alpha=0.5, post_norm=post, eps=1e-2)
    gn = bd.ssm_gated_norm_bwd(y, p["gx"], w["w1"], dy=g2["dx"], groups=groups, gate_first=gate_first, eps=1e-2)
    gs = bd.ssm_gated_scan_bwd(n1, p["ga"], p["gx"], log_a, p["z"], dy=gn["dx"], lengths=lens, h0=h0, dh_last=dh,
                               ckpt=ck)
    g1 = bd.ssm_residual_norm_bwd(p["x"], r1, w["w0"], dy=gs["dx"], dres_out=g2["dres"])
    grads = {"x": g1["dx"], "res": g1["dres"], "ga": gs["dga"], "gx": gs["dgx"] + gn["dz"], "z": gs["dz"],
             "log_a": gs["dlog_a"], "h0": gs["dh0"], "w0": g1["dw_pre"], "w1": gn["dw"], "w2": g2["dw_pre"],
             "w3": g2["dw_post"]}
    leaves = {**p, **w, "log_a": log_a, "h0": h0}
    for n, g in grads.items():
        size = leaves[n].abs() if n == "log_a" else torch.ones_like(g)
        v = torch.sign(g) * size
        old, num = leaves[n].clone(), []
        for h in (1e-2, 5e-3):
            leaves[n].copy_(old + h * v)
            up, step = loss(), leaves[n].double()
            leaves[n].copy_(old - h * v)
            down, step = loss(), step - leaves[n].double()
            num.append((up - down) / (2 * h))
        leaves[n].copy_(old)
        ana = float((g.double() * (step / 1e-2)).sum())
        # The loss sums 4e4 terms of 1 with errors of 1e-6 each: 2e-4, in a difference over 1e-2 0.03, and 4/3 of that
        # here, where both differences are joined so that h^4 is left of the step: 3e-8 of the derivative at most by the
        # same differences in 64 bits.  (Along the gradient itself, whose largest values move z by 0.4, these are off by
        # up to 0.4%.)
        num = (4 * num[1] - num[0]) / 3
        print("  %s: %.6g, by differences %.6g" % (n, ana, num), flush=True)
        assert abs(ana) > 20.0, n
        assert abs(num - ana) <= 0.15 + 1e-3 * abs(ana), (n, num, ana)
