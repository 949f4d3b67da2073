"""ctypes marshalling for the C ABI of ``libssm_scan.so`` (see include/ssm_scan.h).

Argument checks here only concern the Python side (tensor device, dtype,
contiguity, shapes); the library validates again before any HIP call and every
non-OK status becomes an ``SsmError``.
"""
import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm_scan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_OK = 0

_lib = None


class SsmError(RuntimeError):
    def __init__(self, fn, status, detail):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {detail}")


def lib():
    """The loaded ``libssm_scan.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m selective_scan_amd.build` "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, sz, fp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    L.ssm_abi_version.argtypes, L.ssm_abi_version.restype = [], i
    L.ssm_status_string.argtypes, L.ssm_status_string.restype = [i], ctypes.c_char_p
    L.ssm_last_error.argtypes, L.ssm_last_error.restype = [], ctypes.c_char_p
    L.ssm_scan_workspace_size.argtypes, L.ssm_scan_workspace_size.restype = [i, i, i, i], sz
    L.ssm_scan_fwd.argtypes = [i, i, i, i, i] + [vp] * 10 + [vp, sz, vp]
    L.ssm_scan_fwd.restype = i
    L.ssm_scan_fwd_noalloc.argtypes = [i, i, i, i, i] + [vp] * 10 + [vp]
    L.ssm_scan_fwd_noalloc.restype = i
    L.ssm_scan3_workspace_size.argtypes, L.ssm_scan3_workspace_size.restype = [i, i, i, i], sz
    L.ssm_scan3_fwd.argtypes = [i, i, i, i, i] + [vp] * 14 + [vp, sz, vp]
    L.ssm_scan3_fwd.restype = i
    L.ssm_scan_fwd_ex.argtypes = [i, i, i, i, i, i, vp, i] + [vp] * 10 + [vp, sz, vp]
    L.ssm_scan_fwd_ex.restype = i
    L.ssm_step_ex.argtypes = [i, i, i, i, i, vp, i] + [fp] + [vp] * 8 + [vp]
    L.ssm_step_ex.restype = i
    L.ssm_scan_bwd_workspace_size.argtypes, L.ssm_scan_bwd_workspace_size.restype = [i, i, i, i], sz
    L.ssm_scan_bwd.argtypes = [i, i, i, i, i] + [vp] * 18 + [vp, sz, vp]
    L.ssm_scan_bwd.restype = i
    L.ssm_ssd_workspace_size.argtypes, L.ssm_ssd_workspace_size.restype = [i] * 6, sz
    L.ssm_ssd_fwd.argtypes = [i] * 7 + [vp] * 10 + [vp, sz, vp]
    L.ssm_ssd_fwd.restype = i
    L.ssm_step.argtypes = [i, i, i, i] + [fp] + [vp] * 8 + [vp]
    L.ssm_step.restype = i
    L.ssm_ssd_step.argtypes = [i, i, i, i, i] + [fp] + [vp] * 8 + [vp]
    L.ssm_ssd_step.restype = i
    L.ssm_step3.argtypes = [i, i, i, i] + [fp] + [vp] * 12 + [vp]
    L.ssm_step3.restype = i
    f = ctypes.c_float
    L.ssm_linattn_workspace_size.argtypes, L.ssm_linattn_workspace_size.restype = [i] * 7, sz
    L.ssm_linattn_fwd.argtypes = [i] * 7 + [vp] * 4 + [f] + [vp] * 5 + [vp, sz, vp]
    L.ssm_linattn_fwd.restype = i
    L.ssm_linattn_bwd_workspace_size.argtypes, L.ssm_linattn_bwd_workspace_size.restype = [i] * 7, sz
    L.ssm_linattn_bwd.argtypes = [i] * 7 + [vp] * 4 + [f] + [vp] * 8 + [vp, sz, vp]
    L.ssm_linattn_bwd.restype = i
    L.ssm_linattn_step.argtypes = [i] * 6 + [vp] * 5 + [f] + [vp] * 3
    L.ssm_linattn_step.restype = i
    L.ssm_group_norm_workspace_size.argtypes, L.ssm_group_norm_workspace_size.restype = [i] * 5, sz
    L.ssm_group_norm_fwd.argtypes = [i] * 6 + [vp] * 4 + [f] + [vp] * 3 + [vp, sz, vp]
    L.ssm_group_norm_fwd.restype = i
    L.ssm_group_norm_bwd_workspace_size.argtypes, L.ssm_group_norm_bwd_workspace_size.restype = [i] * 5, sz
    L.ssm_group_norm_bwd.argtypes = [i] * 6 + [vp] * 11 + [vp, sz, vp]
    L.ssm_group_norm_bwd.restype = i
    L.ssm_glr_workspace_size.argtypes, L.ssm_glr_workspace_size.restype = [i] * 3, sz
    L.ssm_glr_fwd.argtypes = [i] * 5 + [vp] * 11 + [vp, sz, vp]
    L.ssm_glr_fwd.restype = i
    L.ssm_glr_bwd_workspace_size.argtypes, L.ssm_glr_bwd_workspace_size.restype = [i] * 3, sz
    L.ssm_glr_bwd.argtypes = [i] * 5 + [vp] * 16 + [vp, sz, vp]
    L.ssm_glr_bwd.restype = i
    L.ssm_glr_step.argtypes = [i] * 4 + [vp] * 9
    L.ssm_glr_step.restype = i
    d = ctypes.c_double
    L.ssm_add_norm_fwd.argtypes = [i] * 5 + [vp] * 4 + [f, d] + [vp] * 6
    L.ssm_add_norm_fwd.restype = i
    L.ssm_add_norm_bwd_workspace_size.argtypes, L.ssm_add_norm_bwd_workspace_size.restype = [i] * 4, sz
    L.ssm_add_norm_bwd.argtypes = [i] * 5 + [vp] * 6 + [d] + [vp] * 5 + [vp, sz, vp]
    L.ssm_add_norm_bwd.restype = i
    L.ssm_dropout_blocks.argtypes, L.ssm_dropout_blocks.restype = [i, i], ctypes.c_ulonglong
    L.ssm_dropout.argtypes = [i] * 3 + [vp, d] + [vp] * 3
    L.ssm_dropout.restype = i
    L.ssm_diag_valu_rate.argtypes, L.ssm_diag_valu_rate.restype = [i, i, i, vp, vp], i
    L.ssm_diag_stream_scale.argtypes, L.ssm_diag_stream_scale.restype = [vp, sz, ctypes.c_float, vp], i
    L.ssm_diag_linattn_plan.argtypes, L.ssm_diag_linattn_plan.restype = [i] * 8 + [ctypes.POINTER(i)], i
    L.ssm_diag_copy.argtypes, L.ssm_diag_copy.restype = [vp, vp, sz, vp], i
    _lib = L
    return _lib


# ------------------------------------------------------------------ helpers
def _io_code(t):
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError(f"io tensors must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtype, device, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device, stream):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Allocation context for a call launched on ``stream``: tensors this binding
    allocates (outputs, workspace) are taken from the caching allocator on the
    launch stream itself, so a block freed on return (the workspace) is only handed
    out again to work queued after these kernels on that stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raise(fn, status):
    L = lib()
    raise SsmError(fn, status, L.ssm_last_error().decode())


# ------------------------------------------------------------------ Mamba-1
def ssm_scan_workspace_size(B, L, D, N):
    return int(lib().ssm_scan_workspace_size(B, L, D, N))


SSM_DISC = {"euler": 0, "zoh": 1}


def ssm_scan_fwd(x, delta, A, Bm, Cm, D=None, z=None, h0=None, *, y=None, h_final=None,
                 workspace=None, stream=None, want_final_state=True):
    """Mamba-1 selective scan. x, delta, z: [B, L, D]; Bm, Cm: [B, L, N] (bf16 or fp32);
    A: [D, N], D: [D], h0: [B, D, N] fp32. Returns (y, h_final) (h_final None if not wanted)."""
    return _scan_fwd("ssm_scan_fwd", x, delta, A, Bm, Cm, D, z, h0, y, h_final, workspace, stream,
                     want_final_state, None)


def ssm_scan_fwd_noalloc(x, delta, A, Bm, Cm, D=None, z=None, h0=None, *, y, h_final=None, stream=None):
    """``ssm_scan_fwd`` on the library's fixed per-GPU scratch (no workspace, no
    allocation here or in the library): the caller passes every output tensor.
    Calls that may overlap on one GPU race on the shared scratch."""
    Bb, L, Dd = x.shape
    N = A.shape[1]
    dev, io = x.device, x.dtype
    for t, nm, shp, dt, req in ((x, "x", (Bb, L, Dd), io, True), (delta, "delta", (Bb, L, Dd), io, True),
                                (A, "A", (Dd, N), torch.float32, True), (Bm, "Bm", (Bb, L, N), io, True),
                                (Cm, "Cm", (Bb, L, N), io, True), (D, "D", (Dd,), torch.float32, False),
                                (z, "z", (Bb, L, Dd), io, False), (h0, "h0", (Bb, Dd, N), torch.float32, False),
                                (y, "y", (Bb, L, Dd), io, True),
                                (h_final, "h_final", (Bb, Dd, N), torch.float32, False)):
        _check(t, nm, shp, dt, dev, required=req)
    st = lib().ssm_scan_fwd_noalloc(Bb, L, Dd, N, _io_code(x), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm),
                                    _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_final), _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_scan_fwd_noalloc", st)
    return y, h_final


def ssm_scan_fwd_ex(x, delta, A, Bm, Cm, D=None, z=None, h0=None, *, disc="euler", delta_bias=None,
                    delta_softplus=False, y=None, h_final=None, workspace=None, stream=None,
                    want_final_state=True):
    """``ssm_scan_fwd`` with disc = "euler" | "zoh" (exact zero-order hold) and
    Delta = [softplus](delta + delta_bias) inside the kernels (delta_bias: [D] fp32)."""
    return _scan_fwd("ssm_scan_fwd_ex", x, delta, A, Bm, Cm, D, z, h0, y, h_final, workspace, stream,
                     want_final_state, (SSM_DISC[disc], delta_bias, bool(delta_softplus)))


def _scan_fwd(fn, x, delta, A, Bm, Cm, D, z, h0, y, h_final, workspace, stream, want_final_state, ex):
    Bb, L, Dd = x.shape
    N = A.shape[1]
    dev, io = x.device, x.dtype
    _check(delta, "delta", (Bb, L, Dd), io, dev)
    _check(A, "A", (Dd, N), torch.float32, dev)
    _check(Bm, "Bm", (Bb, L, N), io, dev)
    _check(Cm, "Cm", (Bb, L, N), io, dev)
    _check(D, "D", (Dd,), torch.float32, dev, required=False)
    _check(z, "z", (Bb, L, Dd), io, dev, required=False)
    _check(h0, "h0", (Bb, Dd, N), torch.float32, dev, required=False)
    _check(x, "x", (Bb, L, Dd), io, dev)
    need = ssm_scan_workspace_size(Bb, L, Dd, N)
    with _on(stream):
        if y is None:
            y = torch.empty((Bb, L, Dd), dtype=io, device=dev)
        if want_final_state and h_final is None:
            h_final = torch.empty((Bb, Dd, N), dtype=torch.float32, device=dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(y, "y", (Bb, L, Dd), io, dev)
    _check(h_final, "h_final", (Bb, Dd, N), torch.float32, dev, required=False)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(h0), _ptr(y),
            _ptr(h_final), _ptr(workspace), wbytes, _stream(dev, stream))
    if ex is None:
        st = lib().ssm_scan_fwd(Bb, L, Dd, N, _io_code(x), *args)
    else:
        disc, bias, sp = ex
        _check(bias, "delta_bias", (Dd,), torch.float32, dev, required=False)
        st = lib().ssm_scan_fwd_ex(Bb, L, Dd, N, _io_code(x), disc, _ptr(bias), int(sp), *args)
    if st != SSM_OK:
        _raise(fn, st)
    return y, h_final


def ssm_scan3_workspace_size(B, L, D, N):
    return int(lib().ssm_scan3_workspace_size(B, L, D, N))


def ssm_scan3_fwd(x, delta, lam, Are, theta, Bm, Cm, D=None, z=None, h0=None, x_prev=None, B_prev=None, *,
                  y=None, h_final=None, workspace=None, stream=None, want_final_state=True):
    """Mamba-3 scan. x, delta, lam, z: [B, L, D]; Bm, Cm: [B, L, N] (bf16 or fp32); Are,
    theta: [D, N] fp32; D: [D]; h0: [B, D, N, 2] fp32 (real, imaginary); x_prev [B, D] and
    B_prev [B, N]: the token before the sequence. Returns (y, h_final [B, D, N, 2])."""
    Bb, L, Dd = x.shape
    N = Are.shape[1]
    dev, io = x.device, x.dtype
    for t, nm, shp, dt, req in ((x, "x", (Bb, L, Dd), io, True), (delta, "delta", (Bb, L, Dd), io, True),
                                (lam, "lam", (Bb, L, Dd), io, True), (Are, "Are", (Dd, N), torch.float32, True),
                                (theta, "theta", (Dd, N), torch.float32, True), (Bm, "Bm", (Bb, L, N), io, True),
                                (Cm, "Cm", (Bb, L, N), io, True), (D, "D", (Dd,), torch.float32, False),
                                (z, "z", (Bb, L, Dd), io, False), (h0, "h0", (Bb, Dd, N, 2), torch.float32, False),
                                (x_prev, "x_prev", (Bb, Dd), io, False), (B_prev, "B_prev", (Bb, N), io, False)):
        _check(t, nm, shp, dt, dev, required=req)
    need = ssm_scan3_workspace_size(Bb, L, Dd, N)
    with _on(stream):
        if y is None:
            y = torch.empty((Bb, L, Dd), dtype=io, device=dev)
        if want_final_state and h_final is None:
            h_final = torch.empty((Bb, Dd, N, 2), dtype=torch.float32, device=dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(y, "y", (Bb, L, Dd), io, dev)
    _check(h_final, "h_final", (Bb, Dd, N, 2), torch.float32, dev, required=False)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssm_scan3_fwd(Bb, L, Dd, N, _io_code(x), _ptr(x), _ptr(delta), _ptr(lam), _ptr(Are), _ptr(theta),
                             _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(h0), _ptr(x_prev), _ptr(B_prev), _ptr(y),
                             _ptr(h_final), _ptr(workspace), wbytes, _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_scan3_fwd", st)
    return y, h_final


def ssm_scan_bwd_workspace_size(B, L, D, N):
    return int(lib().ssm_scan_bwd_workspace_size(B, L, D, N))


def ssm_scan_bwd(x, delta, A, Bm, Cm, dy, D=None, z=None, h0=None, dh_final=None, *,
                 want_dh0=True, out=None, workspace=None, stream=None):
    """Gradient of ``ssm_scan_fwd`` for l = sum(dy * y) + sum(dh_final * h_final).

    Inputs as for ``ssm_scan_fwd``; dy: [B, L, D] io dtype; dh_final: [B, D, N] fp32
    or None. Returns a dict with dx, ddelta [B, L, D]; dA [D, N] fp32; dBm, dCm
    [B, L, N]; dD [D] fp32 (None without D); dz [B, L, D] (None without z); dh0
    [B, D, N] fp32 (None unless want_dh0). ``out`` may supply any of these tensors."""
    Bb, L, Dd = x.shape
    N = A.shape[1]
    dev, io = x.device, x.dtype
    _check(x, "x", (Bb, L, Dd), io, dev)
    _check(delta, "delta", (Bb, L, Dd), io, dev)
    _check(A, "A", (Dd, N), torch.float32, dev)
    _check(Bm, "Bm", (Bb, L, N), io, dev)
    _check(Cm, "Cm", (Bb, L, N), io, dev)
    _check(dy, "dy", (Bb, L, Dd), io, dev)
    _check(D, "D", (Dd,), torch.float32, dev, required=False)
    _check(z, "z", (Bb, L, Dd), io, dev, required=False)
    _check(h0, "h0", (Bb, Dd, N), torch.float32, dev, required=False)
    _check(dh_final, "dh_final", (Bb, Dd, N), torch.float32, dev, required=False)
    shapes = dict(dx=((Bb, L, Dd), io), ddelta=((Bb, L, Dd), io), dA=((Dd, N), torch.float32),
                  dBm=((Bb, L, N), io), dCm=((Bb, L, N), io), dD=((Dd,), torch.float32),
                  dz=((Bb, L, Dd), io), dh0=((Bb, Dd, N), torch.float32))
    wanted = dict(dD=D is not None, dz=z is not None, dh0=want_dh0)
    g = dict(out or {})
    need = ssm_scan_bwd_workspace_size(Bb, L, Dd, N)
    with _on(stream):
        for k, (shp, dt) in shapes.items():
            if not wanted.get(k, True):
                g[k] = None
                continue
            if g.get(k) is None:
                g[k] = torch.empty(shp, dtype=dt, device=dev)
            _check(g[k], k, shp, dt, dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssm_scan_bwd(Bb, L, Dd, N, _io_code(x), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm),
                            _ptr(Cm), _ptr(D), _ptr(z), _ptr(h0), _ptr(dy), _ptr(dh_final),
                            *(_ptr(g[k]) for k in ("dx", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "dh0")),
                            _ptr(workspace), wbytes, _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_scan_bwd", st)
    return g


# ------------------------------------------------------------------ SSD
def ssm_ssd_workspace_size(B, L, H, P, N, chunk=0):
    return int(lib().ssm_ssd_workspace_size(B, L, H, P, N, chunk))


def ssm_ssd_fwd(x, delta, A, Bm, Cm, D=None, z=None, h0=None, *, chunk=0, y=None,
                h_final=None, workspace=None, stream=None, want_final_state=True):
    """Mamba-2 SSD chunked scan. x, z: [B, L, H, P]; delta: [B, L, H]; Bm, Cm: [B, L, N];
    A, D: [H] fp32; h0: [B, H, N, P] fp32. Returns (y, h_final)."""
    Bb, L, H, P = x.shape
    N = Bm.shape[2]
    dev, io = x.device, x.dtype
    _check(x, "x", (Bb, L, H, P), io, dev)
    _check(delta, "delta", (Bb, L, H), io, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(Bm, "Bm", (Bb, L, N), io, dev)
    _check(Cm, "Cm", (Bb, L, N), io, dev)
    _check(D, "D", (H,), torch.float32, dev, required=False)
    _check(z, "z", (Bb, L, H, P), io, dev, required=False)
    _check(h0, "h0", (Bb, H, N, P), torch.float32, dev, required=False)
    need = ssm_ssd_workspace_size(Bb, L, H, P, N, chunk)
    with _on(stream):
        if y is None:
            y = torch.empty((Bb, L, H, P), dtype=io, device=dev)
        if want_final_state and h_final is None:
            h_final = torch.empty((Bb, H, N, P), dtype=torch.float32, device=dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(y, "y", (Bb, L, H, P), io, dev)
    _check(h_final, "h_final", (Bb, H, N, P), torch.float32, dev, required=False)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssm_ssd_fwd(Bb, L, H, P, N, int(chunk), _io_code(x), _ptr(x), _ptr(delta), _ptr(A),
                           _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_final),
                           _ptr(workspace), wbytes, _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_ssd_fwd", st)
    return y, h_final


# ------------------------------------------------------------------ decode
def ssm_step(state, x, delta, A, Bm, Cm, D=None, z=None, *, y=None, stream=None):
    """One decode step. state: [B, D, N] fp32 (updated in place); x, delta, z: [B, D];
    Bm, Cm: [B, N]; A: [D, N]; D: [D]. Returns y [B, D]."""
    return _step("ssm_step", state, x, delta, A, Bm, Cm, D, z, y, stream, None)


def ssm_step_ex(state, x, delta, A, Bm, Cm, D=None, z=None, *, disc="euler", delta_bias=None,
                delta_softplus=False, y=None, stream=None):
    """``ssm_step`` with the options of ``ssm_scan_fwd_ex``."""
    return _step("ssm_step_ex", state, x, delta, A, Bm, Cm, D, z, y, stream,
                 (SSM_DISC[disc], delta_bias, bool(delta_softplus)))


def _step(fn, state, x, delta, A, Bm, Cm, D, z, y, stream, ex):
    Bb, Dd, N = state.shape
    dev, io = x.device, x.dtype
    _check(state, "state", (Bb, Dd, N), torch.float32, dev)
    _check(x, "x", (Bb, Dd), io, dev)
    _check(delta, "delta", (Bb, Dd), io, dev)
    _check(A, "A", (Dd, N), torch.float32, dev)
    _check(Bm, "Bm", (Bb, N), io, dev)
    _check(Cm, "Cm", (Bb, N), io, dev)
    _check(D, "D", (Dd,), torch.float32, dev, required=False)
    _check(z, "z", (Bb, Dd), io, dev, required=False)
    if y is None:
        with _on(stream):
            y = torch.empty((Bb, Dd), dtype=io, device=dev)
    _check(y, "y", (Bb, Dd), io, dev)
    args = (_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(y),
            _stream(dev, stream))
    if ex is None:
        st = lib().ssm_step(Bb, Dd, N, _io_code(x), *args)
    else:
        disc, bias, sp = ex
        _check(bias, "delta_bias", (Dd,), torch.float32, dev, required=False)
        st = lib().ssm_step_ex(Bb, Dd, N, _io_code(x), disc, _ptr(bias), int(sp), *args)
    if st != SSM_OK:
        _raise(fn, st)
    return y


def ssm_ssd_step(state, x, delta, A, Bm, Cm, D=None, z=None, *, y=None, stream=None):
    """One Mamba-2 decode step. state: [B, H, N, P] fp32 (updated in place); x, z: [B, H, P];
    delta: [B, H]; Bm, Cm: [B, N]; A: [H]; D: [H]. Returns y [B, H, P]."""
    Bb, H, N, P = state.shape
    dev, io = x.device, x.dtype
    _check(state, "state", (Bb, H, N, P), torch.float32, dev)
    _check(x, "x", (Bb, H, P), io, dev)
    _check(delta, "delta", (Bb, H), io, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(Bm, "Bm", (Bb, N), io, dev)
    _check(Cm, "Cm", (Bb, N), io, dev)
    _check(D, "D", (H,), torch.float32, dev, required=False)
    _check(z, "z", (Bb, H, P), io, dev, required=False)
    if y is None:
        with _on(stream):
            y = torch.empty((Bb, H, P), dtype=io, device=dev)
    _check(y, "y", (Bb, H, P), io, dev)
    st = lib().ssm_ssd_step(Bb, H, P, N, _io_code(x), _ptr(state), _ptr(x), _ptr(delta), _ptr(A),
                            _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(y), _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_ssd_step", st)
    return y


def ssm_step3(state, x, delta, lam, Are, theta, Bm, Cm, D=None, z=None, x_prev=None, B_prev=None, *, y=None,
              stream=None):
    """One Mamba-3 decode step. state: [B, D, N, 2] fp32 (real, imaginary; updated in
    place); x, delta, lam, z: [B, D]; Bm, Cm: [B, N]; Are, theta: [D, N] fp32; D: [D];
    x_prev [B, D] and B_prev [B, N]: the previous token. Returns y [B, D]."""
    Bb, Dd, N, two = state.shape
    dev, io = x.device, x.dtype
    _check(state, "state", (Bb, Dd, N, 2), torch.float32, dev)
    for t, nm, shp, dt, req in ((x, "x", (Bb, Dd), io, True), (delta, "delta", (Bb, Dd), io, True),
                                (lam, "lam", (Bb, Dd), io, True), (Are, "Are", (Dd, N), torch.float32, True),
                                (theta, "theta", (Dd, N), torch.float32, True), (Bm, "Bm", (Bb, N), io, True),
                                (Cm, "Cm", (Bb, N), io, True), (D, "D", (Dd,), torch.float32, False),
                                (z, "z", (Bb, Dd), io, False), (x_prev, "x_prev", (Bb, Dd), io, False),
                                (B_prev, "B_prev", (Bb, N), io, False)):
        _check(t, nm, shp, dt, dev, required=req)
    if y is None:
        with _on(stream):
            y = torch.empty((Bb, Dd), dtype=io, device=dev)
    _check(y, "y", (Bb, Dd), io, dev)
    st = lib().ssm_step3(Bb, Dd, N, _io_code(x), _ptr(state), _ptr(x), _ptr(delta), _ptr(lam), _ptr(Are),
                         _ptr(theta), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(x_prev), _ptr(B_prev), _ptr(y),
                         _stream(dev, stream))
    if st != SSM_OK:
        _raise("ssm_step3", st)
    return y


# ------------------------------------------------------------------ linear attention
class _LinattnNorm(ctypes.Structure):
    """ssm_linattn_norm_t"""
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


def _fits(t, name, shape, dtype, device, required=True):
    """``_check``, and the tensor's address (None without one), at the cost of a few attribute
    reads: a decode step's calls take about as long as its kernels."""
    if t is None and not required:
        return None
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    _check(t, name, shape, dtype, device, required)
    return t.data_ptr()


# the current stream's handle without a Stream object around it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Launch:
    """Makes the tensors' device current where it is not, and gives the stream's handle."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError(f"the tensors are on {device}, not on a GPU")
        self.other = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        self.handle = _raw_stream(device.index) if stream is None else stream.cuda_stream

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _norm_arg(eps, weight, bias, z, HV, shape, io, dev):
    """The norm argument of the linear attention calls (None without norm_eps)."""
    if eps is None:
        if weight is not None or bias is not None or z is not None:
            raise ValueError("norm_weight, norm_bias and z need norm_eps")
        return None
    return ctypes.byref(_LinattnNorm(_fits(weight, "norm_weight", (HV,), torch.float32, dev, False),
                                     _fits(bias, "norm_bias", (HV,), torch.float32, dev, False),
                                     _fits(z, "z", shape, io, dev, False), float(eps)))


def _space(need, workspace, dev):
    """A workspace of ``need`` bytes: (tensor, address, size)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _linattn_dims(q, v):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q and v must be [B, L, heads, dim], got {tuple(q.shape)} and {tuple(v.shape)}")
    return (*q.shape, v.shape[2], v.shape[3])


def ssm_linattn_workspace_size(B, L, H, G, K, V, io=SSM_BF16):
    return int(lib().ssm_linattn_workspace_size(B, L, H, G, K, V, io))


def ssm_linattn_fwd(q, k, v, log_decay, *, scale=None, seqlens=None, h0=None, norm_eps=None, norm_weight=None,
                    norm_bias=None, z=None, o=None, h_final=None, workspace=None, stream=None,
                    want_final_state=True):
    """Linear attention with a decay per head. q, k: [B, L, G, K]; v: [B, L, H, V] (bf16 or
    fp32; G divides H); log_decay: [H] fp32, <= 0; scale: K ** -0.5 by default; seqlens: [B]
    int32, rows past a length are padding (o is 0 there); h0: [B, H, K, V] fp32. With
    ``norm_eps`` o goes through the per-head group norm (norm_weight, norm_bias: [H * V]
    fp32) and the gate silu(z). Returns (o [B, L, H, V], h_final [B, H, K, V])."""
    B, L, G, K, H, V = _linattn_dims(q, v)
    dev, io = q.device, q.dtype
    code = _io_code(q)
    qk, ov, st = (B, L, G, K), (B, L, H, V), (B, H, K, V)
    p = (_fits(q, "q", qk, io, dev), _fits(k, "k", qk, io, dev), _fits(v, "v", ov, io, dev),
         _fits(log_decay, "log_decay", (H,), torch.float32, dev))
    lens = _fits(seqlens, "seqlens", (B,), torch.int32, dev, False)
    h0p = _fits(h0, "h0", st, torch.float32, dev, False)
    norm = _norm_arg(norm_eps, norm_weight, norm_bias, z, H * V, ov, io, dev)
    need = lib().ssm_linattn_workspace_size(B, L, H, G, K, V, code)
    with _on(stream):
        if o is None:
            o = torch.empty(ov, dtype=io, device=dev)
        if want_final_state and h_final is None:
            h_final = torch.empty(st, dtype=torch.float32, device=dev)
        workspace, wp, wbytes = _space(need, workspace, dev)
    op, hp = _fits(o, "o", ov, io, dev), _fits(h_final, "h_final", st, torch.float32, dev, False)
    with _Launch(dev, stream) as s:
        rc = lib().ssm_linattn_fwd(B, L, H, G, K, V, code, *p, max(K, 1) ** -0.5 if scale is None else scale, lens, h0p, norm,
                                   op, hp, wp, wbytes, s)
    if rc != SSM_OK:
        _raise("ssm_linattn_fwd", rc)
    return o, h_final


def ssm_linattn_bwd_workspace_size(B, L, H, G, K, V, io=SSM_BF16):
    return int(lib().ssm_linattn_bwd_workspace_size(B, L, H, G, K, V, io))


def ssm_linattn_bwd(q, k, v, log_decay, dout, *, scale=None, seqlens=None, h0=None, dh_final=None, want_dh0=True,
                    out=None, workspace=None, stream=None):
    """Gradient of ``ssm_linattn_fwd`` (without norm) for l = sum(dout * o) + sum(dh_final *
    h_final). Inputs as for ``ssm_linattn_fwd``; dout: [B, L, H, V]; dh_final: [B, H, K, V]
    fp32 or None. Returns a dict with dq, dk [B, L, G, K], dv [B, L, H, V] (0 at padding) and
    dh0 [B, H, K, V] fp32 (None unless want_dh0). ``out`` may supply any of these tensors."""
    B, L, G, K, H, V = _linattn_dims(q, v)
    dev, io = q.device, q.dtype
    code = _io_code(q)
    qk, ov, st = (B, L, G, K), (B, L, H, V), (B, H, K, V)
    p = (_fits(q, "q", qk, io, dev), _fits(k, "k", qk, io, dev), _fits(v, "v", ov, io, dev),
         _fits(log_decay, "log_decay", (H,), torch.float32, dev))
    dp = _fits(dout, "dout", ov, io, dev)
    lens = _fits(seqlens, "seqlens", (B,), torch.int32, dev, False)
    h0p = _fits(h0, "h0", st, torch.float32, dev, False)
    tp = _fits(dh_final, "dh_final", st, torch.float32, dev, False)
    g, gp = dict(out or {}), []
    need = lib().ssm_linattn_bwd_workspace_size(B, L, H, G, K, V, code)
    with _on(stream):
        for n, shape, dt in (("dq", qk, io), ("dk", qk, io), ("dv", ov, io), ("dh0", st, torch.float32)):
            if n == "dh0" and not want_dh0:
                g[n] = None
            elif g.get(n) is None:
                g[n] = torch.empty(shape, dtype=dt, device=dev)
            gp.append(_fits(g[n], n, shape, dt, dev, n != "dh0"))
        workspace, wp, wbytes = _space(need, workspace, dev)
    with _Launch(dev, stream) as s:
        rc = lib().ssm_linattn_bwd(B, L, H, G, K, V, code, *p, max(K, 1) ** -0.5 if scale is None else scale, lens, h0p, dp, tp,
                                   *gp, wp, wbytes, s)
    if rc != SSM_OK:
        _raise("ssm_linattn_bwd", rc)
    return g


def ssm_linattn_step(state, q, k, v, log_decay, *, scale=None, norm_eps=None, norm_weight=None, norm_bias=None,
                     z=None, o=None, stream=None):
    """One decode step of ``ssm_linattn_fwd``. state: [B, H, K, V] fp32 (updated in place);
    q, k: [B, G, K]; v, z: [B, H, V]; log_decay: [H]; norm arguments as there. Returns o
    [B, H, V]."""
    if state.dim() != 4 or q.dim() != 3:
        raise ValueError(f"state must be [B, H, K, V] and q [B, G, K], got {tuple(state.shape)} and {tuple(q.shape)}")
    B, H, K, V = state.shape
    G = q.shape[1]
    dev, io = q.device, q.dtype
    code = _io_code(q)
    qk, ov = (B, G, K), (B, H, V)
    p = (_fits(state, "state", (B, H, K, V), torch.float32, dev), _fits(q, "q", qk, io, dev),
         _fits(k, "k", qk, io, dev), _fits(v, "v", ov, io, dev),
         _fits(log_decay, "log_decay", (H,), torch.float32, dev))
    norm = _norm_arg(norm_eps, norm_weight, norm_bias, z, H * V, ov, io, dev)
    if o is None:
        with _on(stream):
            o = torch.empty(ov, dtype=io, device=dev)
    op = _fits(o, "o", ov, io, dev)
    with _Launch(dev, stream) as s:
        rc = lib().ssm_linattn_step(B, H, G, K, V, code, *p, max(K, 1) ** -0.5 if scale is None else scale, norm, op, s)
    if rc != SSM_OK:
        _raise("ssm_linattn_step", rc)
    return o


# ------------------------------------------------------------------ group norm
SSM_ACT = {"none": 0, "silu": 1}


def _norm_dims(x):
    """(M, S, C) of x [M, C] (one position per sample) or [M, S, C]."""
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [M, C] or [M, S, C], got shape {tuple(x.shape)}")
    return (x.shape[0], 1, x.shape[1]) if x.dim() == 2 else tuple(x.shape)


def ssm_group_norm_workspace_size(M, S, C, G, io=SSM_BF16):
    return int(lib().ssm_group_norm_workspace_size(M, S, C, G, io))


def ssm_group_norm_fwd(x, groups, weight=None, bias=None, z=None, *, eps=1e-5, act="none", y=None, mean=None,
                       rstd=None, workspace=None, stream=None):
    """Group norm, channels last: y = act((x - mean) rstd weight + bias) [silu(z)]. x, z: [M, S, C]
    (statistics over the S positions and a group's C / groups channels) or [M, C] (S = 1), bf16
    or fp32; weight, bias: [C] fp32; act: "none" | "silu"; y may be x. Returns (y, mean, rstd),
    mean and rstd [M, groups] fp32."""
    M, S, C = _norm_dims(x)
    dev, io, G, act = x.device, x.dtype, int(groups), SSM_ACT[act]
    code, shape = _io_code(x), x.shape
    p = (_fits(x, "x", shape, io, dev), _fits(weight, "weight", (C,), torch.float32, dev, False),
         _fits(bias, "bias", (C,), torch.float32, dev, False), _fits(z, "z", shape, io, dev, False))
    need = lib().ssm_group_norm_workspace_size(M, S, C, G, code)
    with _on(stream):
        if y is None:
            y = torch.empty(shape, dtype=io, device=dev)
        if mean is None:
            mean = torch.empty((M, G), dtype=torch.float32, device=dev)
        if rstd is None:
            rstd = torch.empty((M, G), dtype=torch.float32, device=dev)
        workspace, wp, wbytes = _space(need, workspace, dev)
    out = (_fits(y, "y", shape, io, dev), _fits(mean, "mean", (M, G), torch.float32, dev),
           _fits(rstd, "rstd", (M, G), torch.float32, dev))
    with _Launch(dev, stream) as s:
        rc = lib().ssm_group_norm_fwd(M, S, C, G, code, act, *p, eps, *out, wp, wbytes, s)
    if rc != SSM_OK:
        _raise("ssm_group_norm_fwd", rc)
    return y, mean, rstd


def ssm_group_norm_bwd_workspace_size(M, S, C, G, io=SSM_BF16):
    return int(lib().ssm_group_norm_bwd_workspace_size(M, S, C, G, io))


def ssm_group_norm_bwd(x, groups, mean, rstd, dy, weight=None, bias=None, z=None, *, act="none", want_affine=True,
                       out=None, workspace=None, stream=None):
    """Gradient of ``ssm_group_norm_fwd`` for l = sum(dy * y), from its inputs and its mean and
    rstd. Returns a dict with dx, dweight, dbias [C] fp32 (None unless want_affine), dz (None
    without z). ``out`` may supply any of these tensors."""
    M, S, C = _norm_dims(x)
    dev, io, G, act = x.device, x.dtype, int(groups), SSM_ACT[act]
    code, shape, f32 = _io_code(x), x.shape, torch.float32
    p = (_fits(x, "x", shape, io, dev), _fits(weight, "weight", (C,), f32, dev, False),
         _fits(bias, "bias", (C,), f32, dev, False), _fits(z, "z", shape, io, dev, False),
         _fits(mean, "mean", (M, G), f32, dev), _fits(rstd, "rstd", (M, G), f32, dev), _fits(dy, "dy", shape, io, dev))
    g, gp = dict(out or {}), []
    need = lib().ssm_group_norm_bwd_workspace_size(M, S, C, G, code)
    with _on(stream):
        for n, sh, dt, wanted in (("dx", shape, io, True), ("dweight", (C,), f32, want_affine),
                                  ("dbias", (C,), f32, want_affine), ("dz", shape, io, z is not None)):
            if not wanted:
                g[n] = None
            elif g.get(n) is None:
                g[n] = torch.empty(sh, dtype=dt, device=dev)
            gp.append(_fits(g[n], n, sh, dt, dev, wanted))
        workspace, wp, wbytes = _space(need, workspace, dev)
    with _Launch(dev, stream) as s:
        rc = lib().ssm_group_norm_bwd(M, S, C, G, code, act, *p, *gp, wp, wbytes, s)
    if rc != SSM_OK:
        _raise("ssm_group_norm_bwd", rc)
    return g


# ------------------------------------------------------------------ gated linear recurrence
def _run(fn, dev, stream, *args):
    """fn(*args, stream handle) with the tensors' device current; its status."""
    if dev.type == "cuda" and torch.cuda.current_device() == dev.index:
        return fn(*args, _raw_stream(dev.index) if stream is None else stream.cuda_stream)
    with _Launch(dev, stream) as s:
        return fn(*args, s)


def _new(like, shape, dtype, stream):
    """An output tensor: ``like``'s kind where no shape is given (a contiguous tensor of the shape
    and type wanted: the cheapest to make), on the launch stream."""
    if stream is None:
        return torch.empty_like(like) if shape is None else torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return _new(like, shape, dtype, None)


def _output(t, name, like, shape, dtype, stream, whole=False):
    """(tensor, address): the caller's output after checks, or a new one (``whole``: as ``like``)."""
    if t is None:
        t = _new(like, None if whole else shape, dtype, stream)
        return t, t.data_ptr()
    return t, _fits(t, name, shape, dtype, like.device)


def _outputs(given, like, stream, wanted):
    """(dict, addresses) of a gradient's outputs (name, shape, dtype, whether wanted): the caller's
    or new ones, None where not wanted."""
    g, at = dict(given or {}), []
    plain, own = like.is_contiguous(), like.shape
    for name, shape, dtype, want in wanted:
        if want:
            g[name], p = _output(g.get(name), name, like, shape, dtype, stream,
                                 plain and dtype is like.dtype and shape == own)
            at.append(p)
        else:
            g[name] = None
            at.append(None)
    return g, at


SSM_GLR_FORM = {"decay": 0, "convex": 1}
SSM_GLR_STATE_STEPS = 128


def _strided(t, name, shape, dtype, device):
    """(address, row stride) of a tensor whose rows may be further apart than they are long (a
    slice of a projection's output): [B, L, D] or [B, D] with neighbouring channels neighbours in
    memory and every row as far from the next."""
    D = shape[-1]
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return t.data_ptr(), D
        ld, rows, even = D, 1, D == 1 or t.stride(-1) == 1
        for n, s in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):  # the inner rows first
            if n > 1:
                if rows == 1:
                    ld = s
                even, rows = even and s == ld * rows, rows * n
        if even and D <= ld < 2 ** 31:
            return t.data_ptr(), ld
        if t.numel():
            raise ValueError(f"{name} must have adjacent channels and evenly spaced rows, got strides {t.stride()}")
    _check(t, name, shape, dtype, device)
    return t.data_ptr(), D


def _glr_inputs(x, r, i, A, z, form):
    """(form code, io code, addresses of x, r, i, A, z and the row strides) after checks."""
    form, code, dev, io, shape = SSM_GLR_FORM[form], _io_code(x), x.device, x.dtype, x.shape
    decay, D = form == 0, shape[-1]
    if decay != (A is not None) or decay != (i is not None):
        raise ValueError("i and A are given exactly with form 'decay'")
    xp, lx = _strided(x, "x", shape, io, dev)
    rp, lr = _strided(r, "r", shape, io, dev)
    ip, li = _strided(i, "i", shape, io, dev) if decay else (None, D)
    zp, lz = (None, D) if z is None else _strided(z, "z", shape, io, dev)
    Ap = _fits(A, "A", (D,), torch.float32, dev) if decay else None
    ld = None if lx == lr == li == lz == D else (ctypes.c_int * 4)(lx, lr, li, lz)
    return form, code, (xp, rp, ip, Ap, zp, ld)


def ssm_glr_workspace_size(B, L, D):
    return int(lib().ssm_glr_workspace_size(B, L, D))


def ssm_glr_fwd(x, r, i=None, A=None, z=None, *, form="decay", seqlens=None, h0=None, y=None, h_final=None,
                states=None, workspace=None, stream=None, want_final_state=True, want_states=False):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t, y = h [silu(z)]. form "decay": a = exp(A
    sigmoid(r)), u = sqrt(1 - a^2) sigmoid(i) x; "convex" (without i and A): a = 1 - sigmoid(r), u =
    sigmoid(r) x. x, r, i, z: [B, L, D] bf16 or fp32, rows may be strided (slices of a projection);
    A: [D] fp32, in [-2^100, 0]; seqlens: [B] int32, rows past a length are padding (y is 0 there); h0: [B, D]
    fp32. Returns (y [B, L, D], h_final [B, D] fp32, states), the last with ``want_states``: the
    state entering every 128th step, [B, ceil(L / 128), D] fp32, for ``ssm_glr_bwd``."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, L, D], got {tuple(x.shape)}")
    B, L, D = x.shape
    dev, io, f32 = x.device, x.dtype, torch.float32
    form, code, p = _glr_inputs(x, r, i, A, z, form)
    lens, h0p = _fits(seqlens, "seqlens", (B,), torch.int32, dev, False), _fits(h0, "h0", (B, D), f32, dev, False)
    n = -(-L // SSM_GLR_STATE_STEPS)
    need = lib().ssm_glr_workspace_size(B, L, D)
    hp = sp = None
    y, yp = _output(y, "y", x, (B, L, D), io, stream, x.is_contiguous())
    if want_final_state or h_final is not None:
        h_final, hp = _output(h_final, "h_final", x, (B, D), f32, stream)
    if want_states or states is not None:
        states, sp = _output(states, "states", x, (B, n, D), f32, stream)
    if workspace is None and need > 0:
        workspace = _new(x, (need,), torch.uint8, stream)
    workspace, wp, wbytes = _space(0, workspace, dev)
    rc = _run(lib().ssm_glr_fwd, dev, stream, B, L, D, code, form, *p, lens, h0p, yp, hp, sp, wp, wbytes)
    if rc != SSM_OK:
        _raise("ssm_glr_fwd", rc)
    return y, h_final, states


def ssm_glr_bwd_workspace_size(B, L, D):
    return int(lib().ssm_glr_bwd_workspace_size(B, L, D))


def ssm_glr_bwd(x, r, states, dy, i=None, A=None, z=None, *, form="decay", seqlens=None, dh_final=None, want_dh0=True,
                out=None, workspace=None, stream=None):
    """Gradient of ``ssm_glr_fwd`` for l = sum(dy * y) + sum(dh_final * h_final), from its inputs
    and the ``states`` it returned. dy: [B, L, D]; dh_final: [B, D] fp32 or None. Returns a dict
    with dx, dr, di, dz [B, L, D] (0 at padding; di, dz None without i, z), dA [D] fp32 (None
    without A) and dh0 [B, D] fp32 (None unless want_dh0). ``out`` may supply any of these."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, L, D], got {tuple(x.shape)}")
    B, L, D = x.shape
    dev, io, f32, shape = x.device, x.dtype, torch.float32, tuple(x.shape)
    form, code, p = _glr_inputs(x, r, i, A, z, form)
    lens = _fits(seqlens, "seqlens", (B,), torch.int32, dev, False)
    ins = (_fits(states, "states", (B, -(-L // SSM_GLR_STATE_STEPS), D), f32, dev), _fits(dy, "dy", shape, io, dev),
           _fits(dh_final, "dh_final", (B, D), f32, dev, False))
    need = lib().ssm_glr_bwd_workspace_size(B, L, D)
    g, gp = _outputs(out, x, stream, (("dx", shape, io, True), ("dr", shape, io, True), ("di", shape, io, i is not None),
                                      ("dA", (D,), f32, A is not None), ("dz", shape, io, z is not None),
                                      ("dh0", (B, D), f32, want_dh0)))
    if workspace is None and need > 0:
        workspace = _new(x, (need,), torch.uint8, stream)
    workspace, wp, wbytes = _space(0, workspace, dev)
    rc = _run(lib().ssm_glr_bwd, dev, stream, B, L, D, code, form, *p, lens, *ins, *gp, wp, wbytes)
    if rc != SSM_OK:
        _raise("ssm_glr_bwd", rc)
    return g


def ssm_glr_step(state, x, r, i=None, A=None, z=None, *, form="decay", y=None, stream=None):
    """One decode step of ``ssm_glr_fwd``. state: [B, D] fp32 (updated in place); x, r, i, z: [B, D],
    rows may be strided; A: [D]. Returns y [B, D]."""
    if x.dim() != 2:
        raise ValueError(f"x must be [B, D], got {tuple(x.shape)}")
    B, D = x.shape
    dev, io = x.device, x.dtype
    form, code, p = _glr_inputs(x, r, i, A, z, form)
    sp = _fits(state, "state", (B, D), torch.float32, dev)
    y, yp = _output(y, "y", x, (B, D), io, stream, x.is_contiguous())
    rc = _run(lib().ssm_glr_step, dev, stream, B, D, code, form, sp, *p, yp)
    if rc != SSM_OK:
        _raise("ssm_glr_step", rc)
    return y


# ------------------------------------------------------------------ residual add, norm, dropout
SSM_NORM = {"layer": 0, "rms": 1}


def _rows_dims(t, name):
    """(M, C) of a tensor of rows [..., C]."""
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be [..., C], got shape {tuple(t.shape)}")
    C = t.shape[-1]
    return t.numel() // C, C


def ssm_add_norm_fwd(x, residual=None, weight=None, bias=None, *, eps=1e-5, norm="layer", p=0.0, rng=None, y=None,
                     sum=None, mean=None, rstd=None, want_sum=True, stream=None):
    """s = residual + dropout(x), then y = norm(s) weight + bias over the last dimension: norm
    "layer" ((s - mean) rstd) or "rms" (s rstd). x: [..., C] bf16 or fp32; residual: the same shape,
    fp32 or x's type; weight, bias: [C] fp32; p, rng: as for ``ssm_dropout``. y may be x, sum may be
    residual. Returns (y, sum, mean, rstd): sum in the residual's type (x itself where nothing is
    added or dropped and y is not written over it; None unless want_sum), mean (None for "rms") and rstd [...] fp32."""
    M, C = _rows_dims(x, "x")
    dev, io, f32, shape = x.device, x.dtype, torch.float32, x.shape
    code, kind = _io_code(x), SSM_NORM[norm]
    given = residual if residual is not None else sum
    res = io if given is None else given.dtype
    rcode = code if given is None else _io_code(given)
    xp = _fits(x, "x", shape, io, dev)
    ep = None if residual is None else _fits(residual, "residual", shape, res, dev)
    wp = None if weight is None else _fits(weight, "weight", (C,), f32, dev)
    bp = None if bias is None else _fits(bias, "bias", (C,), f32, dev)
    rp = _fits(rng, "rng", (2,), torch.int64, dev) if p != 0.0 else None
    # the sum is x, unless y is written over it
    same = sum is None and residual is None and p == 0.0 and (y is None or y.data_ptr() != xp)
    sp = mp = None
    y, yp = _output(y, "y", x, shape, io, stream, True)
    if sum is not None or (want_sum and not same):
        sum, sp = _output(sum, "sum", x if residual is None else residual, shape, res, stream, residual is not None)
    if mean is not None or kind == 0:
        mean, mp = _output(mean, "mean", x, shape[:-1], f32, stream)
    rstd, dp = _output(rstd, "rstd", x, shape[:-1], f32, stream)
    rc = _run(lib().ssm_add_norm_fwd, dev, stream, M, C, code, rcode, kind, xp, ep, wp, bp, eps, p, rp, yp, sp, mp, dp)
    if rc != SSM_OK:
        _raise("ssm_add_norm_fwd", rc)
    return y, (x if same and want_sum else sum), mean, rstd


def ssm_add_norm_bwd_workspace_size(M, C, io=SSM_BF16, res=SSM_F32):
    return int(lib().ssm_add_norm_bwd_workspace_size(M, C, io, res))


def ssm_add_norm_bwd(sum, mean, rstd, dy, weight=None, dsum=None, *, norm="layer", p=0.0, rng=None, want_dx=True,
                     want_dresidual=True, want_dweight=True, want_dbias=True, out=None, workspace=None, stream=None):
    """Gradient of ``ssm_add_norm_fwd`` from the sum, mean and rstd it returned. dy: [..., C];
    dsum: the gradient that the residual stream brings from later layers, in sum's type, or None.
    Returns a dict with dx (dy's type), dresidual (sum's type; may be dsum), dweight and dbias [C]
    fp32, None where not wanted. ``out`` may supply any of these tensors."""
    M, C = _rows_dims(dy, "dy")
    dev, io, f32, shape = dy.device, dy.dtype, torch.float32, dy.shape
    code, kind, res, rcode = _io_code(dy), SSM_NORM[norm], sum.dtype, _io_code(sum)
    ins = (_fits(sum, "sum", shape, res, dev), _fits(weight, "weight", (C,), f32, dev, False),
           _fits(mean, "mean", shape[:-1], f32, dev, kind == 0), _fits(rstd, "rstd", shape[:-1], f32, dev),
           _fits(dy, "dy", shape, io, dev), _fits(dsum, "dsum", shape, res, dev, False))
    rp = _fits(rng, "rng", (2,), torch.int64, dev) if p != 0.0 else None
    need = lib().ssm_add_norm_bwd_workspace_size(M, C, code, rcode) if want_dweight or want_dbias else 0
    g, gp = _outputs(out, dy, stream, (("dx", shape, io, want_dx), ("dresidual", shape, res, want_dresidual),
                                       ("dweight", (C,), f32, want_dweight), ("dbias", (C,), f32, want_dbias)))
    if workspace is None and need > 0:
        workspace = _new(dy, (need,), torch.uint8, stream)
    workspace, wp, wbytes = _space(0, workspace, dev)
    rc = _run(lib().ssm_add_norm_bwd, dev, stream, M, C, code, rcode, kind, *ins, p, rp, *gp, wp, wbytes)
    if rc != SSM_OK:
        _raise("ssm_add_norm_bwd", rc)
    return g


def ssm_dropout_blocks(M, C):
    """Counter values that dropout of [M, C] uses: the next call's offset is this much further."""
    return int(lib().ssm_dropout_blocks(M, C))


def ssm_dropout(x, p, rng=None, *, y=None, stream=None):
    """Dropout of x [..., C] (bf16 or fp32) whose mask comes from a counter: each element is 0 with
    probability p (a multiple of 2^-16), else scaled by 1 / (1 - p). rng: [2] int64 on x's device,
    (seed, offset), read when the kernel runs. On dy with the same rng it is the gradient. y may be x."""
    M, C = _rows_dims(x, "x")
    dev, io, shape, code = x.device, x.dtype, x.shape, _io_code(x)
    xp, rp = _fits(x, "x", shape, io, dev), _fits(rng, "rng", (2,), torch.int64, dev) if p != 0.0 else None
    y, yp = _output(y, "y", x, shape, io, stream, True)
    rc = _run(lib().ssm_dropout, dev, stream, M, C, code, xp, p, rp, yp)
    if rc != SSM_OK:
        _raise("ssm_dropout", rc)
    return y


# ------------------------------------------------------------------ diagnostics
def ssm_diag_valu_rate(mode, out, iters, stream=None):
    """VALU issue-rate probe (mode 0 exp, 1 fma, 2 exp:fma 1:3, 3 sin, 4 cos); ``out`` is an fp32
    tensor of blocks * 256 elements. Returns the number of ops it issues."""
    blocks = out.numel() // 256
    st = lib().ssm_diag_valu_rate(int(mode), blocks, int(iters), _ptr(out), _stream(out.device, stream))
    if st != SSM_OK:
        _raise("ssm_diag_valu_rate", st)
    return blocks * 256 * 32 * int(iters)


def ssm_diag_stream_scale(t, s, stream=None):
    """t *= s in place on a contiguous fp32 tensor (the pure-streaming floor)."""
    _check(t, "t", tuple(t.shape), torch.float32, t.device)
    st = lib().ssm_diag_stream_scale(_ptr(t), t.numel(), float(s), _stream(t.device, stream))
    if st != SSM_OK:
        _raise("ssm_diag_stream_scale", st)


def ssm_diag_copy(src, dst, stream=None):
    """dst = src for contiguous fp32 tensors of the same shape (the copy kernel the HBM
    byte counters are calibrated with)."""
    _check(src, "src", tuple(src.shape), torch.float32, src.device)
    _check(dst, "dst", tuple(src.shape), torch.float32, src.device)
    st = lib().ssm_diag_copy(_ptr(src), _ptr(dst), src.numel(), _stream(src.device, stream))
    if st != SSM_OK:
        _raise("ssm_diag_copy", st)


def ssm_diag_linattn_plan(B, L, H, G, K, V, io=SSM_BF16, gradient=False):
    """How ``ssm_linattn_fwd`` or its gradient cuts a sequence: dict(chunks, supers, per_super,
    pieces, per_piece, together); counts of 64-step chunks, see ``include/ssm_scan.h``."""
    plan = (ctypes.c_int * 6)()
    st = lib().ssm_diag_linattn_plan(B, L, H, G, K, V, io, int(gradient), plan)
    if st != SSM_OK:
        _raise("ssm_diag_linattn_plan", st)
    return dict(zip(("chunks", "supers", "per_super", "pieces", "per_piece", "together"), plan))
