"""Calls at the edges of what linear attention and the norm with rotation accept:
no heads, counts that leave 64 bits, more workgroups than a launch holds
(nothing is launched)."""
from selective_state_space_84_amd import binding as bd

P0 = 0x7F0000000000
MB = 1 << 20


def test_norm_gradient_of_no_heads_reads_nothing(lib):
    """Without heads no frequencies are needed, and without weight gradients nothing is left to launch."""
    rc = lib.ssm_qk_norm_rope_bwd(None, None, None, None, None, None, None, None, None, None, None, None, 2, 10, 0, 0, 64,
                                  64, 0, 0, 1e-6, 0, 1, None, 0, None)
    assert rc == bd.SSM_OK


def _attn(lib, b, L, H, M, grad=False, dk=64, dv=64, dtype=1):
    if grad:
        return lib.ssm_linear_attn_bwd(*[None] * 12, b, L, H, M, dk, dv, 0, 0, 0, 0.125, dtype, None, 0, None)
    return lib.ssm_linear_attn_fwd(*[None] * 8, b, L, H, M, dk, dv, 0, 0, 0, 0.125, dtype, None, 0, None)


def test_counts_without_heads_stay_in_range(lib):
    """Without query heads nothing bounded the key/value heads or the steps: products of them left 64 bits."""
    for grad in (False, True):
        assert _attn(lib, 2, 10, 0, 1 << 60, grad) == bd.SSM_ERR_BAD_DIM
        assert _attn(lib, 2, 10, 0, (1 << 15) + 1, grad) == bd.SSM_ERR_BAD_DIM
        assert _attn(lib, 1 << 40, 1 << 30, 0, 1, grad) == bd.SSM_ERR_BAD_DIM
        assert _attn(lib, 1 << 30, 1 << 30, 0, 1 << 15, grad) == bd.SSM_ERR_BAD_DIM
    assert lib.ssm_linear_attn_update(*[None] * 7, 2, 2, 0, 1 << 60, 64, 64, 0, 0, 0, 0.125, 1, None) == \
        bd.SSM_ERR_BAD_DIM


def test_gradient_of_shared_heads_without_query_heads_needs_outputs(lib):
    """dk and dv of no query heads are zeros, which somebody has to write."""
    assert _attn(lib, 2, 10, 0, 2, grad=True) == bd.SSM_ERR_NULL_ARG
    assert _attn(lib, 2, 0, 0, 2, grad=True) == bd.SSM_OK
    assert _attn(lib, 2, 10, 0, 2) == bd.SSM_OK
