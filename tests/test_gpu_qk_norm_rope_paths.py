"""Norm of query and key heads with the rotation: calls and launch shapes beside
those of test_gpu_qk_norm_rope.py, against the 64-bit definitions."""
import numpy as np
import pytest

import plain64 as P
from test_gpu_linear_attn import DEV, _np
from test_gpu_qk_norm_rope import _check, _freq, _make

pytestmark = pytest.mark.gpu


def test_gradient_of_no_heads(lib):
    """The weights' gradients are sums over nothing; the frequencies (here absent) are not read."""
    import torch
    from selective_state_space_84_amd import binding
    dw = torch.full((2, 64), float("nan"), device=DEV)
    need = lib.ssm_qk_norm_rope_bwd_workspace_size(2, 10, 0, 0, 64)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    rc = lib.ssm_qk_norm_rope_bwd(None, None, None, None, None, None, None, None, None, None, dw[0].data_ptr(),
                                  dw[1].data_ptr(), 2, 10, 0, 0, 64, 64, 0, 0, 1e-6, 0, 1, ws.data_ptr(), need, None)
    torch.cuda.synchronize()
    assert rc == binding.SSM_OK and not dw.any()
    z = torch.zeros(2, 10, 0, 64, device=DEV)
    g = binding.ssm_qk_norm_rope_bwd(z, None, inv_freq=torch.ones(32, device=DEV), dq_out=z)
    assert g["dq"].shape == z.shape and not g["dwq"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,L,H,M,D,R", [
    (1, 4101, 9, 8, 256, 256),    # forward 2 rounds of one step; gradient 8, and 513 turns on 512 workgroups
    (3, 2801, 40, 24, 64, 32),    # forward 2 rounds of 2 steps; gradient 8 of 2
    (1, 32771, 1, 0, 256, 64),    # 2 rounds of 8 steps, the last turn of 3; gradient 4 or 5 turns a workgroup
    (1, 3001, 20, 4, 80, 48)])    # gradient 2 of 2 steps, 751 turns: 239 workgroups walk two
def test_several_rounds(lib, B, L, H, M, D, R, inter, dtype):
    """Several rounds a workgroup on one set of angles, several turns a workgroup in the gradient, as long prompts and
    training batches run."""
    print("case", B, L, H, M, D, R, inter, dtype, flush=True)
    _check(*_make(B + L, B, L, H, M, D, R, dtype), dtype, 1e-6, inter, D)


@pytest.mark.parametrize("B,L,H,M,D,R", [(1, 4101, 9, 8, 256, 256), (3, 2801, 4, 2, 64, 32), (1, 32771, 1, 1, 64, 64),
                                         (1, 3001, 20, 4, 80, 48), (1, 511, 3, 1, 128, 128), (1, 513, 3, 1, 128, 0)])
def test_weight_gradients_take_every_step_once(lib, B, L, H, M, D, R):
    """dw over all steps, by its norm: a step left out or taken twice shows as 1 / sqrt(steps), 5e-3 at least, where
    sums of at most 170 roundings one after the other are off by 170 * 2^-24 = 1e-5 if all of them go one way."""
    import torch
    from selective_state_space_84_amd import binding
    q, k, wq, wk, f, pos, dq, dk = _make(B + L + 1, B, L, H, M, D, R, "bf16")
    g = binding.ssm_qk_norm_rope_bwd(q, k, wq, wk, f, dq_out=dq, dk_out=dk, positions=pos)
    torch.cuda.synchronize()
    p = pos.cpu().numpy()
    for name, x, w, dy in (("dwq", q, wq, dq), ("dwk", k, wk, dk)):
        ref = P.norm_rope_bwd(_np(x), _np(w), p, _freq(f), 1e-6, False, _np(dy))[1]
        off = np.linalg.norm(_np(g[name]) - ref) / np.linalg.norm(ref)
        print("  %s: %.3g" % (name, off), flush=True)
        assert off < 1e-5
