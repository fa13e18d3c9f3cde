"""ctypes binding of the gfx950 selective-scan library (libssm_scan.so).

Argument marshalling only: the functions here check tensor placement,
allocate outputs or workspace when the caller passes none, and hand raw device
pointers and the current HIP stream to the C ABI declared in
``include/ssm_scan.h``.  Every step of the computation runs in the library's
kernels.  There is no fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm_scan.so")

SSM_DTYPE_F32 = 0
SSM_DTYPE_BF16 = 1
SSM_FLAG_DELTA_SOFTPLUS = 0x1
SSM_FLAG_EXACT_ZOH = 0x2
SSM_FLAG_A_LINEAR_N = 0x4

SSM_OK = 0
SSM_ERR_NULL_ARG = -1
SSM_ERR_BAD_DIM = -2
SSM_ERR_UNSUPPORTED = -3
SSM_ERR_MISALIGNED = -4
SSM_ERR_WORKSPACE = -5
SSM_ERR_HIP = -6
SSM_ERR_ALIAS = -7

# Every symbol the header declares, with its ctypes signature.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_U32 = ctypes.c_uint32
_SZ = ctypes.c_size_t
_F32 = ctypes.c_float


class ScanOpts(ctypes.Structure):
    """Mirror of ssm_scan_opts_t."""
    _fields_ = [("n_split", ctypes.c_int32), ("reserved0", ctypes.c_int32), ("chunk_len", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved1", ctypes.c_uint32), ("dt_bias", ctypes.c_void_p),
                ("ckpt_out", ctypes.c_void_p)]


SIGNATURES = {
    "ssm_abi_version": ([], ctypes.c_int),
    "ssm_strerror": ([ctypes.c_int], ctypes.c_char_p),
    "ssm_scan_fwd_workspace_size": ([_I64, _I64, _I64, _I64], _SZ),
    "ssm_scan_fwd_ex_workspace_size": ([_I64, _I64, _I64, _I64, ctypes.POINTER(ScanOpts)], _SZ),
    "ssm_scan_fwd_plan": ([_I64, _I64, _I64, _I64, ctypes.POINTER(ScanOpts), ctypes.POINTER(_I32),
                           ctypes.POINTER(_I64), ctypes.POINTER(_I64)], ctypes.c_int),
    "ssm_scan_fwd": ([_P] * 10 + [_I64] * 4 + [_I32, _P, _SZ, _P], ctypes.c_int),
    "ssm_scan_fwd_ex": ([_P] * 10 + [_I64] * 4 + [_I32, ctypes.POINTER(ScanOpts), _P, _SZ, _P], ctypes.c_int),
    "ssm_scan_fwd_noalloc": ([_P] * 10 + [_I64] * 4 + [_I32, ctypes.POINTER(ScanOpts), _P], ctypes.c_int),
    "ssm_scan_fwd_noalloc_max_bytes": ([], _SZ),
    "ssm_state_update": ([_P] * 9 + [_I64] * 3 + [_I32, _P], ctypes.c_int),
    "ssm_state_update_ex": ([_P] * 9 + [_I64] * 3 + [_I32, _U32, _P, _P], ctypes.c_int),
    "ssm_scan_bwd_workspace_size": ([_I64, _I64, _I64, _I64], _SZ),
    "ssm_scan_bwd_workspace_size_ex": ([_I64, _I64, _I64, _I64, _I32], _SZ),
    "ssm_scan_ckpt_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "ssm_scan_bwd": ([_P] * 21 + [_I64] * 4 + [_I32, _U32, _P, _SZ, _P], ctypes.c_int),
    "ssm_ssd_fwd": ([_P] * 10 + [_I64] * 6 + [_I32, _U32, _P, _P], ctypes.c_int),
    "ssm_conv1d_fwd": ([_P] * 6 + [_I64] * 4 + [_I32, _I32, _P], ctypes.c_int),
    "ssm_conv1d_update": ([_P] * 5 + [_I64] * 3 + [_I32, _I32, _P], ctypes.c_int),
    "ssm_linear_attn_fwd": ([_P] * 8 + [_I64] * 9 + [_F32, _I32, _P, _SZ, _P], ctypes.c_int),
    "ssm_linear_attn_fwd_workspace_size": ([_I64] * 5 + [_I32], _SZ),
    "ssm_linear_attn_bwd": ([_P] * 12 + [_I64] * 9 + [_F32, _I32, _P, _SZ, _P], ctypes.c_int),
    "ssm_linear_attn_bwd_workspace_size": ([_I64] * 6 + [_I32], _SZ),
    "ssm_linear_attn_update": ([_P] * 7 + [_I64] * 9 + [_F32, _I32, _P], ctypes.c_int),
    "ssm_qk_norm_rope_fwd": ([_P] * 8 + [_I64] * 10 + [_F32, _I32, _I32, _P], ctypes.c_int),
    "ssm_qk_norm_rope_bwd": ([_P] * 12 + [_I64] * 8 + [_F32, _I32, _I32, _P, _SZ, _P], ctypes.c_int),
    "ssm_qk_norm_rope_bwd_workspace_size": ([_I64] * 5, _SZ),
}

_lib = None


class SsmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, strerror(status), status))


def load_library(path: Optional[str] = None):
    """Load libssm_scan.so (built in-tree by build_lib.build()); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libssm_scan.so is not built (%s); run python -m selective_state_space_84_amd.build_lib" % p)
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def abi_version() -> int:
    return load_library().ssm_abi_version()


def strerror(status: int) -> str:
    return load_library().ssm_strerror(status).decode()


def _opts(n_split=0, chunk_len=0, flags=0, dt_bias=None, ckpt_out=None) -> ScanOpts:
    return ScanOpts(n_split, 0, chunk_len, flags, 0, _ptr(dt_bias), _ptr(ckpt_out))


def scan_ckpt_bytes(batch, seqlen, d_inner, d_state) -> int:
    """Bytes of the block-start state checkpoints a forward call can save."""
    n = load_library().ssm_scan_ckpt_bytes(batch, seqlen, d_inner, d_state)
    if n == ctypes.c_size_t(-1).value:
        raise SsmError(SSM_ERR_BAD_DIM, "ssm_scan_ckpt_bytes")
    return n


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr() or None


def _io_dtype(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SSM_DTYPE_BF16
    if t.dtype == torch.float32:
        return SSM_DTYPE_F32
    raise ValueError("io tensors must be bfloat16 or float32, got %s" % t.dtype)


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def scan_plan(batch, seqlen, d_inner, d_state, n_split=0, chunk_len=0, flags=0) -> Tuple[int, int, int]:
    """(n_split, chunk_len, n_chunks) the library launches for these sizes."""
    g = _I32()
    cl = _I64()
    nc = _I64()
    o = _opts(n_split, chunk_len, flags)
    rc = load_library().ssm_scan_fwd_plan(batch, seqlen, d_inner, d_state, ctypes.byref(o), ctypes.byref(g),
                                          ctypes.byref(cl), ctypes.byref(nc))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_scan_fwd_plan")
    return g.value, cl.value, nc.value


def scan_workspace_size(batch, seqlen, d_inner, d_state, n_split=0, chunk_len=0, flags=0) -> int:
    o = _opts(n_split, chunk_len, flags)
    n = load_library().ssm_scan_fwd_ex_workspace_size(batch, seqlen, d_inner, d_state, ctypes.byref(o))
    if n == ctypes.c_size_t(-1).value:
        raise SsmError(SSM_ERR_BAD_DIM, "ssm_scan_fwd_ex_workspace_size")
    return n


def ssm_scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None, *, y=None, h_last=None, want_h_last=True,
                 workspace=None, n_split=0, chunk_len=0, flags=0, dt_bias=None, ckpt_out=None, stream=None):
    """Selective scan over the sequence; returns (y, h_last).

    x, delta, z: (batch, seqlen, d_inner); A: (d_inner, d_state) fp32;
    B, C: (batch, seqlen, d_state); D: (d_inner,) fp32; h0: (batch, d_inner, d_state) fp32.
    io tensors are all bfloat16 or all float32.  Outputs are allocated when not given.
    ckpt_out: optional fp32 buffer of scan_ckpt_bytes() bytes that receives the
    state before every 8-step block (for ssm_scan_bwd(ckpt=...)).
    """
    import torch
    batch, seqlen, d_inner = x.shape
    d_state = A.shape[1]
    dt = _io_dtype(x)
    if y is None:
        y = torch.empty_like(x)
    if h_last is None and want_h_last:
        h_last = torch.empty((batch, d_inner, d_state), dtype=torch.float32, device=x.device)
    ws_bytes = scan_workspace_size(batch, seqlen, d_inner, d_state, n_split, chunk_len, flags)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    ws_have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    o = _opts(n_split, chunk_len, flags, dt_bias, ckpt_out)
    rc = load_library().ssm_scan_fwd_ex(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last),
        batch, seqlen, d_inner, d_state, dt, ctypes.byref(o), _ptr(workspace), ws_have, _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_scan_fwd")
    return y, h_last


def ssm_scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, h0=None, *, y, h_last=None, n_split=0, chunk_len=0,
                         flags=0, dt_bias=None, stream=None):
    """ssm_scan_fwd without a workspace: the library's per-device scratch holds
    the chunk carries and nothing is allocated (y and h_last must be given)."""
    batch, seqlen, d_inner = x.shape
    d_state = A.shape[1]
    o = _opts(n_split, chunk_len, flags, dt_bias, None)
    rc = load_library().ssm_scan_fwd_noalloc(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last),
        batch, seqlen, d_inner, d_state, _io_dtype(x), ctypes.byref(o), _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_scan_fwd_noalloc")
    return y, h_last


def ssm_state_update(h, x_t, delta_t, A, B_t, C_t, D=None, z_t=None, *, y_t=None, flags=0, dt_bias=None,
                     stream=None):
    """One decode step, in place on h (batch, d_inner, d_state) fp32; returns y_t."""
    import torch
    batch, d_inner, d_state = h.shape
    dt = _io_dtype(x_t)
    if y_t is None:
        y_t = torch.empty_like(x_t)
    rc = load_library().ssm_state_update_ex(
        _ptr(h), _ptr(x_t), _ptr(delta_t), _ptr(A), _ptr(B_t), _ptr(C_t), _ptr(D), _ptr(z_t), _ptr(y_t),
        batch, d_inner, d_state, dt, flags, _ptr(dt_bias), _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_state_update")
    return y_t


def scan_bwd_workspace_size(batch, seqlen, d_inner, d_state, ckpt_given=False) -> int:
    """Backward workspace bytes; smaller when the forward call's checkpoints are passed."""
    n = load_library().ssm_scan_bwd_workspace_size_ex(batch, seqlen, d_inner, d_state, 1 if ckpt_given else 0)
    if n == ctypes.c_size_t(-1).value:
        raise SsmError(SSM_ERR_BAD_DIM, "ssm_scan_bwd_workspace_size_ex")
    return n


def ssm_scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, *, dy, dh_last=None, flags=0, dt_bias=None,
                 ckpt=None, want_dh0=True, grads=None, workspace=None, stream=None):
    """Gradient of ssm_scan_fwd for L = sum(dy * y) + sum(dh_last * h_last).

    ckpt: optional checkpoints saved by the forward call (ssm_scan_fwd(ckpt_out=...)).

    Returns a dict with dx, ddelta (w.r.t. the delta argument as passed), dA,
    dB, dC (fp32), and dD, dz, dh0, d_dt_bias when D, z, want_dh0, the softplus
    flag are used.  Outputs are allocated unless given in ``grads``.
    """
    import torch
    batch, seqlen, d_inner = x.shape
    d_state = A.shape[1]
    dt = _io_dtype(x)
    dev = x.device
    g = dict(grads or {})
    f32 = dict(dtype=torch.float32, device=dev)
    if "dx" not in g:
        g["dx"] = torch.empty_like(x)
    if "ddelta" not in g:
        g["ddelta"] = torch.empty_like(x)
    if "dA" not in g:
        g["dA"] = torch.empty((d_inner, d_state), **f32)
    if "dB" not in g:
        g["dB"] = torch.empty((batch, seqlen, d_state), **f32)
    if "dC" not in g:
        g["dC"] = torch.empty((batch, seqlen, d_state), **f32)
    if D is not None and "dD" not in g:
        g["dD"] = torch.empty((d_inner,), **f32)
    if z is not None and "dz" not in g:
        g["dz"] = torch.empty_like(x)
    if want_dh0 and "dh0" not in g:
        g["dh0"] = torch.empty((batch, d_inner, d_state), **f32)
    if (flags & SSM_FLAG_DELTA_SOFTPLUS) and "d_dt_bias" not in g:
        g["d_dt_bias"] = torch.empty((d_inner,), **f32)
    ws_bytes = scan_bwd_workspace_size(batch, seqlen, d_inner, d_state, ckpt_given=ckpt is not None)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ws_have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().ssm_scan_bwd(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(dt_bias), _ptr(dy),
        _ptr(dh_last), _ptr(ckpt), _ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
        _ptr(g.get("dD")), _ptr(g.get("dz")), _ptr(g.get("dh0")), _ptr(g.get("d_dt_bias")), batch, seqlen, d_inner,
        d_state, dt, flags, _ptr(workspace), ws_have, _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_scan_bwd")
    return g


def ssm_ssd_fwd(x, dt, A, B, C, D=None, z=None, h0=None, *, y=None, h_last=None, want_h_last=True, flags=0,
                dt_bias=None, stream=None):
    """Scan with a scalar decay per head (Mamba-2 / SSD form); returns (y, h_last).

    x, z: (batch, seqlen, nheads, 64) bf16; dt: (batch, seqlen, nheads) bf16;
    A, D, dt_bias: (nheads,) fp32; B, C: (batch, seqlen, ngroups, d_state) bf16;
    h0: (batch, nheads, 64, d_state) fp32.
    """
    import torch
    batch, seqlen, nheads, headdim = x.shape
    ngroups, d_state = B.shape[2], B.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if h_last is None and want_h_last:
        h_last = torch.empty((batch, nheads, headdim, d_state), dtype=torch.float32, device=x.device)
    rc = load_library().ssm_ssd_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0),
                                    _ptr(y), _ptr(h_last), batch, seqlen, nheads, headdim, ngroups, d_state,
                                    _io_dtype(x), flags, _ptr(dt_bias), _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_ssd_fwd")
    return y, h_last


def ssm_conv1d_fwd(x, w, bias=None, state_in=None, *, y=None, state_out=None, want_state=True, silu=True,
                   stream=None):
    """Causal depthwise conv1d (+ SiLU); returns (y, state_out).

    x: (batch, seqlen, d_inner) bf16/fp32; w: (d_inner, d_conv) fp32;
    bias: (d_inner,) fp32; state_in / state_out: (batch, d_inner, d_conv-1) fp32.
    """
    import torch
    batch, seqlen, d_inner = x.shape
    d_conv = w.shape[1]
    if y is None:
        y = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty((batch, d_inner, d_conv - 1), dtype=torch.float32, device=x.device)
    rc = load_library().ssm_conv1d_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(state_in), _ptr(y), _ptr(state_out),
                                       batch, seqlen, d_inner, d_conv, _io_dtype(x), 1 if silu else 0,
                                       _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_conv1d_fwd")
    return y, state_out


def ssm_conv1d_update(state, x_t, w, bias=None, *, y_t=None, silu=True, stream=None):
    """One decode step of the conv, in place on state (batch, d_inner, d_conv-1); returns y_t."""
    import torch
    batch, d_inner = x_t.shape
    d_conv = w.shape[1]
    if y_t is None:
        y_t = torch.empty_like(x_t)
    rc = load_library().ssm_conv1d_update(_ptr(state), _ptr(x_t), _ptr(w), _ptr(bias), _ptr(y_t), batch, d_inner,
                                          d_conv, _io_dtype(x_t), 1 if silu else 0, _stream(stream))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_conv1d_update")
    return y_t


def _rows(t, what: str) -> Tuple[Optional[int], int]:
    """(pointer, elements between steps) of a tensor (rows, heads, width) or
    (batch, steps, heads, width) whose steps are evenly spaced dense (heads,
    width) blocks: a dense tensor, or a column range of a wider one."""
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    shape = t.shape
    heads, width = shape[-2:]
    dense = heads * width
    if t.is_contiguous():
        return t.data_ptr() or None, dense
    st = t.stride()
    ok = (st[-1] == 1 or width <= 1) and (st[-2] == width or heads <= 1)
    if len(shape) == 3:
        step = st[0] if shape[0] > 1 else dense
    else:
        batch, steps = shape[:2]
        step = st[1] if steps > 1 else (st[0] if batch > 1 else dense)
        ok = ok and len(shape) == 4 and (batch <= 1 or st[0] == step * steps)
    if not ok or step < dense:
        raise ValueError("%s must hold dense (heads, width) blocks at one step apart" % what)
    return t.data_ptr() or None, step


_no_scope = contextlib.nullcontext()


def _scope(stream, t, *others):
    """Context in which t's device is current, and so is stream (a torch stream
    or a raw handle) when one is given: what is allocated inside belongs to the
    stream that uses it.  Every other tensor must be on t's device."""
    import torch
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensor must live on the GPU")
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError("tensors must be on one device, got %s and %s" % (t.device, o.device))
    if stream is None:
        return _no_scope if torch.cuda.current_device() == dev else torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)  # also makes the stream's device current


def _here(t) -> Optional[int]:
    """Raw handle of the stream that is current on t's device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device()) or None


def _workspace(workspace, need, device, what):
    import torch
    if need == ctypes.c_size_t(-1).value:
        raise SsmError(SSM_ERR_BAD_DIM, what)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _want(t, shape, dtype, what):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError("%s must be %s %s, got %s %s" % (what, tuple(shape), dtype, tuple(t.shape), t.dtype))


def _dense(t, what) -> Optional[int]:
    """_ptr of a tensor that is known to be on the GPU."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr() or None


def _fill(g, names, device):
    """Checks the outputs given in g and allocates the others; names: (name, shape, dtype)."""
    import torch
    if g:
        known = [name for name, _, _ in names]
        for n in g:
            if n not in known:
                raise ValueError("unknown output %s" % n)
    for name, shape, dtype in names:
        t = g.get(name)
        if t is None:
            g[name] = torch.empty(shape, dtype=dtype, device=device)
        else:
            _want(t, shape, dtype, name)


def _attn_shapes(q, k, v, lead):
    """Sizes of q (*lead, nheads, d_k), k (*lead, nheads_kv, d_k), v (*lead, nheads_kv, d_v)."""
    nheads, d_k = q.shape[-2:]
    nheads_kv, d_v = v.shape[-2:]
    if q.dim() != lead + 2:
        raise ValueError("q must have %d axes, got %s" % (lead + 2, tuple(q.shape)))
    rows = q.shape[:lead]
    _want(k, rows + (nheads_kv, d_k), q.dtype, "k")
    _want(v, rows + (nheads_kv, d_v), q.dtype, "v")
    return nheads, nheads_kv, d_k, d_v


def ssm_linear_attn_fwd(q, k, v, log_decay, *, lengths=None, h0=None, scale=None, o=None, h_last=None,
                        want_h_last=True, workspace=None, stream=None):
    """Linear attention with a constant decay per head; returns (o, h_last).

    q: (batch, seqlen, nheads, d_k); k: (batch, seqlen, nheads_kv, d_k);
    v: (batch, seqlen, nheads_kv, d_v), all bfloat16 or all float32, dense or
    column ranges of one wider tensor; log_decay: (nheads,) fp32;
    lengths: (batch,) int32 steps of each row; h0, h_last:
    (batch, nheads, d_v, d_k) fp32; scale defaults to d_k ** -0.5.
    """
    import torch
    nheads, nheads_kv, d_k, d_v = _attn_shapes(q, k, v, 2)
    batch, seqlen = q.shape[:2]
    dt = _io_dtype(q)
    f32 = torch.float32
    st = (batch, nheads, d_v, d_k)
    _want(log_decay, (nheads,), f32, "log_decay")
    _want(lengths, (batch,), torch.int32, "lengths")
    _want(h0, st, f32, "h0")
    _want(o, (batch, seqlen, nheads, d_v), q.dtype, "o")
    _want(h_last, st, f32, "h_last")
    lib = load_library()
    with _scope(stream, q, k, v, log_decay, lengths, h0, o, h_last, workspace):
        if o is None:
            o = torch.empty((batch, seqlen, nheads, d_v), dtype=q.dtype, device=q.device)
        if h_last is None and want_h_last:
            h_last = torch.empty(st, dtype=f32, device=q.device)
        need = lib.ssm_linear_attn_fwd_workspace_size(batch, seqlen, nheads, d_k, d_v, dt)
        workspace, have = _workspace(workspace, need, q.device, "ssm_linear_attn_fwd")
        (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
        rc = lib.ssm_linear_attn_fwd(qp, kp, vp, _ptr(log_decay), _ptr(lengths), _ptr(h0), _ptr(o), _ptr(h_last),
                                     batch, seqlen, nheads, nheads_kv, d_k, d_v, qs, ks, vs,
                                     d_k ** -0.5 if scale is None else scale, dt, _ptr(workspace), have,
                                     _here(q))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_linear_attn_fwd")
    return o, h_last


def ssm_linear_attn_bwd(q, k, v, log_decay, *, do, lengths=None, h0=None, dh_last=None, scale=None, want_dh0=True,
                        grads=None, workspace=None, stream=None):
    """Gradient of ssm_linear_attn_fwd for L = sum(do * o) + sum(dh_last * h_last).

    Returns a dict with dq, dk, dv (io dtype, dense) and, when want_dh0, dh0
    (fp32).  Outputs are allocated unless given in ``grads``.
    """
    import torch
    nheads, nheads_kv, d_k, d_v = _attn_shapes(q, k, v, 2)
    batch, seqlen = q.shape[:2]
    dt = _io_dtype(q)
    f32 = torch.float32
    st = (batch, nheads, d_v, d_k)
    _want(log_decay, (nheads,), f32, "log_decay")
    _want(lengths, (batch,), torch.int32, "lengths")
    _want(h0, st, f32, "h0")
    _want(dh_last, st, f32, "dh_last")
    _want(do, (batch, seqlen, nheads, d_v), q.dtype, "do")
    g = dict(grads or {})
    names = [("dq", q.shape, q.dtype), ("dk", k.shape, q.dtype), ("dv", v.shape, q.dtype)]
    if want_dh0 or "dh0" in g:
        names.append(("dh0", st, f32))
    lib = load_library()
    with _scope(stream, q, k, v, log_decay, lengths, h0, do, dh_last, workspace, *g.values()):
        _fill(g, names, q.device)
        need = lib.ssm_linear_attn_bwd_workspace_size(batch, seqlen, nheads, nheads_kv, d_k, d_v, dt)
        workspace, have = _workspace(workspace, need, q.device, "ssm_linear_attn_bwd")
        (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
        rc = lib.ssm_linear_attn_bwd(qp, kp, vp, _ptr(log_decay), _ptr(lengths), _ptr(h0), _ptr(do), _ptr(dh_last),
                                     _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g.get("dh0")), batch, seqlen,
                                     nheads, nheads_kv, d_k, d_v, qs, ks, vs,
                                     d_k ** -0.5 if scale is None else scale, dt, _ptr(workspace), have,
                                     _here(q))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_linear_attn_bwd")
    return g


def ssm_linear_attn_update(h, q, k, v, log_decay, *, slots=None, scale=None, o=None, stream=None):
    """One decode step, in place on h (n_slots, nheads, d_v, d_k) fp32; returns o (batch, nheads, d_v).

    q: (batch, nheads, d_k); k: (batch, nheads_kv, d_k); v: (batch, nheads_kv,
    d_v); slots: (batch,) int32 places of the requests' states in h (values
    outside h mark unused rows; used values must differ), or None when h holds
    the batch in order.
    """
    import torch
    f32, qt = torch.float32, q.dtype
    batch, nheads, d_k = q.shape
    n_slots, nheads_kv, d_v = h.shape[0], v.shape[1], v.shape[-1]
    # One comparison for the usual case; the checks one by one name what is wrong.
    if not (k.shape == (batch, nheads_kv, d_k) and v.shape == (batch, nheads_kv, d_v) and
            h.shape == (n_slots, nheads, d_v, d_k) and log_decay.shape == (nheads,) and k.dtype is qt and
            v.dtype is qt and h.dtype is f32 and log_decay.dtype is f32 and
            (slots is None or (slots.shape == (batch,) and slots.dtype is torch.int32)) and
            (o is None or (o.shape == (batch, nheads, d_v) and o.dtype is qt))):
        _attn_shapes(q, k, v, 1)
        _want(h, (n_slots, nheads, d_v, d_k), f32, "h")
        _want(log_decay, (nheads,), f32, "log_decay")
        _want(slots, (batch,), torch.int32, "slots")
        _want(o, (batch, nheads, d_v), qt, "o")
        raise ValueError("arguments do not fit together")
    dt = _io_dtype(q)
    with _scope(stream, q, h, slots, k, v, log_decay, o):
        if o is None:
            o = torch.empty((batch, nheads, d_v), dtype=qt, device=q.device)
        (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
        rc = load_library().ssm_linear_attn_update(
            _dense(h, "h"), _dense(slots, "slots"), qp, kp, vp, _dense(log_decay, "log_decay"), _dense(o, "o"), batch,
            n_slots, nheads, nheads_kv, d_k, d_v, qs, ks, vs, d_k ** -0.5 if scale is None else scale, dt, _here(q))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_linear_attn_update")
    return o


def _qk_shapes(q, k):
    batch, seqlen, nheads, headdim = q.shape
    nheads_k = 0 if k is None else k.shape[2]
    _want(k, (batch, seqlen, nheads_k, headdim), q.dtype, "k")
    return batch, seqlen, nheads, nheads_k, headdim


def _qk_params(wq, wk, inv_freq, positions, batch, seqlen, headdim):
    """Checks of the norm weights, frequencies and positions; returns rot_dim."""
    import torch
    f32 = torch.float32
    if wq is not None:
        _want(wq, (headdim,), f32, "wq")
    if wk is not None:
        _want(wk, (headdim,), f32, "wk")
    if positions is not None:
        _want(positions, (batch, seqlen), torch.int64, "positions")
    if inv_freq is None:
        return 0
    n = inv_freq.numel()
    _want(inv_freq, (n,), f32, "inv_freq")
    return 2 * n


def _side(x, out, what):
    """(input, its step, output, its step, output tensor) of q or k; the output is allocated when None."""
    import torch
    if x is None:
        if out is not None:
            raise ValueError("%s_out given without %s" % (what, what))
        return None, 0, None, 0, None
    p, step = _rows(x, what)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        return p, step, out.data_ptr() or None, 0, out
    _want(out, x.shape, x.dtype, what + "_out")
    return (p, step, *_rows(out, what + "_out"), out)


def ssm_qk_norm_rope_fwd(q, k, wq=None, wk=None, inv_freq=None, *, positions=None, eps=1e-6, interleaved=False,
                         q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head, then the rotation of its first
    2 * len(inv_freq) values by position * inv_freq; returns (q_out, k_out).

    q: (batch, seqlen, nheads, headdim), k: (batch, seqlen, nheads_k, headdim)
    or None; wq, wk: (headdim,) fp32 or None for ones; positions:
    (batch, seqlen) int64, or None for the step's index.  q_out and k_out may be q
    and k themselves (in place).
    """
    batch, seqlen, nheads, nheads_k, headdim = _qk_shapes(q, k)
    rot = _qk_params(wq, wk, inv_freq, positions, batch, seqlen, headdim)
    with _scope(stream, q, k, wq, wk, inv_freq, positions, q_out, k_out):
        qp, qs, qo, qos, q_out = _side(q, q_out, "q")
        kp, ks, ko, kos, k_out = _side(k, k_out, "k")
        rc = load_library().ssm_qk_norm_rope_fwd(
            qp, kp, _dense(wq, "wq"), _dense(wk, "wk"), _dense(inv_freq, "inv_freq"), _dense(positions, "positions"),
            qo, ko, batch, seqlen, nheads, nheads_k, headdim, rot, qs, ks, qos, kos, eps, 1 if interleaved else 0,
            _io_dtype(q), _here(q))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_qk_norm_rope_fwd")
    return q_out, k_out


def ssm_qk_norm_rope_bwd(q, k, wq=None, wk=None, inv_freq=None, *, dq_out, dk_out=None, positions=None, eps=1e-6,
                         interleaved=False, want_dw=True, grads=None, workspace=None, stream=None):
    """Gradient of ssm_qk_norm_rope_fwd from its inputs and the gradients of its
    outputs: a dict with dq, dk (dense) and, when want_dw, dwq, dwk (fp32).
    Outputs are allocated unless given in ``grads``."""
    import torch
    batch, seqlen, nheads, nheads_k, headdim = _qk_shapes(q, k)
    rot = _qk_params(wq, wk, inv_freq, positions, batch, seqlen, headdim)
    _want(dq_out, q.shape, q.dtype, "dq_out")
    g = dict(grads or {})
    names = [("dq", q.shape, q.dtype)]
    if want_dw:
        names.append(("dwq", (headdim,), torch.float32))
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out is required with k" if dk_out is None else "dk_out given without k")
    if k is not None:
        _want(dk_out, k.shape, q.dtype, "dk_out")
        names.append(("dk", k.shape, q.dtype))
        if want_dw:
            names.append(("dwk", (headdim,), torch.float32))
    lib = load_library()
    with _scope(stream, q, k, wq, wk, inv_freq, positions, dq_out, dk_out, workspace, *g.values()):
        _fill(g, names, q.device)
        need = 0
        if want_dw:
            need = lib.ssm_qk_norm_rope_bwd_workspace_size(batch, seqlen, nheads, nheads_k, headdim)
        workspace, have = _workspace(workspace, need, q.device, "ssm_qk_norm_rope_bwd")
        qp, qs = _rows(q, "q")
        kp, ks = (None, 0) if k is None else _rows(k, "k")
        rc = lib.ssm_qk_norm_rope_bwd(
            qp, kp, _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(positions), _ptr(dq_out),
            None if k is None else _ptr(dk_out), _ptr(g["dq"]), _ptr(g.get("dk")), _ptr(g.get("dwq")),
            _ptr(g.get("dwk")), batch, seqlen, nheads, nheads_k, headdim, rot, qs, ks, eps, 1 if interleaved else 0,
            _io_dtype(q), _ptr(workspace), have, _here(q))
    if rc != SSM_OK:
        raise SsmError(rc, "ssm_qk_norm_rope_bwd")
    return g
