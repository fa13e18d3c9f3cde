"""Norm of query and key heads with the rotation: calls and launch shapes beside
those of test_gpu_qk_norm_rope.py, against the 64-bit definitions."""
import pytest

from test_gpu_linear_attn import DEV

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
