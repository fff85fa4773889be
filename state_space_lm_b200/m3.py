"""Python binding of the C ABI in ``include/m3.h`` (ctypes).

Argument marshalling only: every step of the scan runs in the CUDA library.
Tensors are torch CUDA tensors (PyTorch supplies device memory and streams);
outputs that the caller does not pass are allocated with ``torch.empty``.
If the library has not been built, every call raises ``RuntimeError`` -- there
is no other implementation behind these names.
"""
import ctypes
import functools
import os

import torch

from .build import LIB

M3_OK, M3_ERR_INVALID_ARG, M3_ERR_UNSUPPORTED, M3_ERR_WORKSPACE, M3_ERR_CUDA, M3_ERR_TIMEOUT = range(6)
M3_F32, M3_BF16 = 0, 1
M3_WS_SISO, M3_WS_MIMO, M3_WS_BWD_SISO, M3_WS_BWD_MIMO = 0, 1, 2, 3

_DTYPE = {torch.float32: M3_F32, torch.bfloat16: M3_BF16}

ABI_FUNCTIONS = (
    "m3_get_limits", "m3_discretize", "m3_rope_bc", "m3_siso_chunked_fwd",
    "m3_mimo_chunked_fwd", "m3_step_decode", "m3_workspace_bytes", "m3_status_string",
    "m3_launch_count", "m3_device_error", "m3_siso_chunked_fwd_noalloc", "m3_mimo_step_decode",
    "m3_step_decode_factored", "m3_chunked_bwd", "m3_selftest_bounded_wait", "m3_debug_fail_next_launches",
    "m3_linattn_chunked_fwd", "m3_linattn_step_decode", "m3_linattn_chunked_bwd", "m3_linattn_workspace_bytes",
    "m3_group_norm_fwd", "m3_group_norm_bwd", "m3_group_norm_workspace_bytes",
)
M3_SELFTEST_SITE = 99
M3_WS_LINATTN_FWD, M3_WS_LINATTN_BWD = 0, 1
M3_WS_NORM_FWD, M3_WS_NORM_BWD = 0, 1
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}

GRAD_FIELDS = ("dx", "ddt", "dA", "dlam", "dtheta", "dB", "dC", "dD", "dW_x", "dW_y",
               "dnormw_B", "dnormw_C", "dbias_B", "dbias_C", "dh0", "dprevBx0", "dangle0")


class M3Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("rank", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("rope_pairs", ctypes.c_int64)]


class BcNorm(ctypes.Structure):
    _fields_ = [("normw_B", ctypes.c_void_p), ("normw_C", ctypes.c_void_p),
                ("bias_B", ctypes.c_void_p), ("bias_C", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in GRAD_FIELDS]


class LinattnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "headdim", "dstate", "ngroups",
                                              "ld_q", "ld_k", "ld_v")]


class LinattnGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dq", "dk", "dv", "ds0")]


class NormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "channels", "ngroups")]


class Limits(ctypes.Structure):
    _fields_ = [("max_dstate", ctypes.c_int64), ("max_headdim", ctypes.c_int64),
                ("max_state_elems", ctypes.c_int64), ("max_rank", ctypes.c_int64)]


_lib = None
_VP = ctypes.c_void_p


def library_path():
    return LIB


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError("the CUDA library %s is missing: run `python -m state_space_lm_b200.build`"
                           % LIB)
    L = ctypes.CDLL(LIB)
    L.m3_get_limits.restype = Limits
    L.m3_get_limits.argtypes = []
    L.m3_status_string.restype = ctypes.c_char_p
    L.m3_status_string.argtypes = [ctypes.c_int]
    L.m3_workspace_bytes.restype = ctypes.c_size_t
    L.m3_workspace_bytes.argtypes = [ctypes.c_int, Dims, ctypes.c_int]
    L.m3_launch_count.restype = ctypes.c_uint64
    L.m3_launch_count.argtypes = []
    L.m3_device_error.restype = ctypes.c_int
    L.m3_device_error.argtypes = [_VP, ctypes.POINTER(ctypes.c_int)]
    L.m3_discretize.restype = ctypes.c_int
    L.m3_discretize.argtypes = [_VP, _VP, _VP, Dims, _VP, _VP, _VP, _VP]
    L.m3_rope_bc.restype = ctypes.c_int
    L.m3_rope_bc.argtypes = [_VP, _VP, ctypes.c_int, _VP, _VP, _VP, ctypes.POINTER(BcNorm), Dims,
                             _VP, _VP, _VP, _VP]
    L.m3_siso_chunked_fwd.restype = ctypes.c_int
    L.m3_siso_chunked_fwd.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                      ctypes.POINTER(BcNorm), _VP, _VP, _VP, Dims, _VP, _VP, _VP,
                                      _VP, _VP, ctypes.c_size_t, _VP]
    L.m3_mimo_chunked_fwd.restype = ctypes.c_int
    L.m3_mimo_chunked_fwd.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                      ctypes.c_int, ctypes.POINTER(BcNorm), _VP, _VP, _VP, Dims,
                                      _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]
    L.m3_step_decode.restype = ctypes.c_int
    L.m3_step_decode.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                 ctypes.POINTER(BcNorm), Dims, _VP, _VP, _VP, _VP, _VP]
    for fn in (L.m3_mimo_step_decode, L.m3_step_decode_factored):
        fn.restype = ctypes.c_int
    L.m3_mimo_step_decode.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                      ctypes.POINTER(BcNorm), Dims, _VP, _VP, _VP, _VP, _VP]
    L.m3_step_decode_factored.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                          ctypes.POINTER(BcNorm), Dims, _VP, _VP, _VP, _VP, _VP, _VP]
    L.m3_selftest_bounded_wait.restype = ctypes.c_int
    L.m3_selftest_bounded_wait.argtypes = [_VP]
    L.m3_debug_fail_next_launches.restype = None
    L.m3_debug_fail_next_launches.argtypes = [ctypes.c_int]
    L.m3_chunked_bwd.restype = ctypes.c_int
    L.m3_chunked_bwd.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                 ctypes.POINTER(BcNorm), _VP, _VP, _VP, Dims, _VP, _VP, _VP, _VP,
                                 ctypes.POINTER(Grads), _VP, ctypes.c_size_t, _VP]
    i, sz, fl = ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L.m3_linattn_chunked_fwd.restype = i
    L.m3_linattn_chunked_fwd.argtypes = [_VP, _VP, _VP, i, _VP, fl, _VP, _VP, LinattnDims, _VP, _VP, _VP, sz, _VP]
    L.m3_linattn_step_decode.restype = i
    L.m3_linattn_step_decode.argtypes = [_VP, _VP, _VP, i, _VP, fl, LinattnDims, _VP, _VP, _VP]
    L.m3_linattn_chunked_bwd.restype = i
    L.m3_linattn_chunked_bwd.argtypes = [_VP, _VP, _VP, i, _VP, fl, _VP, _VP, LinattnDims, _VP, _VP,
                                         ctypes.POINTER(LinattnGrads), _VP, sz, _VP]
    L.m3_linattn_workspace_bytes.restype = sz
    L.m3_linattn_workspace_bytes.argtypes = [i, LinattnDims, i]
    L.m3_group_norm_fwd.restype = i
    L.m3_group_norm_fwd.argtypes = [_VP, i, _VP, _VP, _VP, i, fl, NormDims, _VP, _VP, _VP, _VP, sz, _VP]
    L.m3_group_norm_bwd.restype = i
    L.m3_group_norm_bwd.argtypes = [_VP, _VP, i, _VP, _VP, _VP, i, _VP, _VP, NormDims, _VP, _VP, _VP, _VP, _VP, sz,
                                    _VP]
    L.m3_group_norm_workspace_bytes.restype = sz
    L.m3_group_norm_workspace_bytes.argtypes = [i, NormDims, i]
    _lib = L
    return L


def status_string(status):
    return lib().m3_status_string(int(status)).decode()


def launch_count():
    return int(lib().m3_launch_count())


def device_error(stream=None, with_site=False):
    """Synchronise the stream and return the device-side error status
    (M3_OK, or M3_ERR_TIMEOUT when a bounded wait inside a kernel gave up);
    with_site=True also returns the recorded wait site."""
    site = ctypes.c_int(0)
    st = int(lib().m3_device_error(_stream(stream), ctypes.byref(site)))
    return (st, site.value) if with_site else st


def selftest_bounded_wait(stream=None):
    """Enqueue the timeout-path self-test (one bounded wait that runs out after
    about a second); read the outcome with device_error()."""
    _check(lib().m3_selftest_bounded_wait(_stream(stream)), "m3_selftest_bounded_wait")


def debug_fail_next_launches(n):
    """Failure injection for tests: the next n library calls that pass their
    argument checks fail with M3_ERR_CUDA (raised as M3Error here) and
    launch nothing.  n <= 0 turns it off."""
    lib().m3_debug_fail_next_launches(int(n))


def limits():
    l = lib().m3_get_limits()
    return dict(max_dstate=l.max_dstate, max_headdim=l.max_headdim,
                max_state_elems=l.max_state_elems, max_rank=l.max_rank)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _expect(where, dev, name, t, numel, dtype, required=True):
    """The library sees only pointers and the sizes in m3_dims, so the binding
    checks each tensor against those sizes (element count, dtype, device)
    before the call: a tensor shorter than the sizes say would otherwise be
    read or written past its end."""
    if t is None:
        if required:
            raise ValueError("%s: %s is required" % (where, name))
        return
    if t.numel() != numel:
        raise ValueError("%s: %s has %d elements (shape %s), the sizes need %d"
                         % (where, name, t.numel(), tuple(t.shape), numel))
    if t.dtype != dtype:
        raise ValueError("%s: %s is %s, expected %s" % (where, name, t.dtype, dtype))
    if t.device != dev:
        raise ValueError("%s: %s is on %s, expected %s" % (where, name, t.device, dev))


def _io_dtype(where, t):
    if t.dtype not in _DTYPE:
        raise ValueError("%s: x, B, C must be float32 or bfloat16, got %s" % (where, t.dtype))
    return t.dtype


def _expect_norm(where, dev, norm, H, R, N):
    if norm is None:
        return
    for k in ("normw_B", "normw_C"):
        _expect(where, dev, k, norm.get(k), N, torch.float32, required=False)
    for k in ("bias_B", "bias_C"):
        _expect(where, dev, k, norm.get(k), H * R * N, torch.float32, required=False)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _norm(norm):
    if norm is None:
        return None, ()
    keep = tuple(norm.get(k) for k in ("normw_B", "normw_C", "bias_B", "bias_C"))
    s = BcNorm(*[_ptr(k) for k in keep], float(norm.get("eps", 1e-5)))
    return ctypes.byref(s), keep + (s,)


def _check(rc, where):
    if rc != M3_OK:
        raise M3Error(rc, where)


def workspace_bytes(which, dims, dtype):
    return int(lib().m3_workspace_bytes(int(which), dims, int(dtype)))


def discretize(dt, A, lam, out=None, stream=None):
    """S1: alpha, beta, gamma (Bt,T,H) fp32."""
    Bt, T, H = dt.shape
    al, be, ga = out if out is not None else tuple(torch.empty_like(dt) for _ in range(3))
    w, f, n, dev = "m3_discretize", torch.float32, Bt * T * H, dt.device
    for name, t in (("dt", dt), ("lam", lam), ("alpha", al), ("beta", be), ("gamma", ga)):
        _expect(w, dev, name, t, n, f)
    _expect(w, dev, "A", A, H, f)
    d = Dims(Bt, T, H, 1, 2, 1, 1, 0, 0)
    _check(lib().m3_discretize(_ptr(dt), _ptr(A), _ptr(lam), d, _ptr(al), _ptr(be), _ptr(ga),
                               _stream(stream)), "m3_discretize")
    return al, be, ga


def rope_bc(B, C, theta, dt, angle0=None, norm=None, out=None, stream=None):
    """S2: B_rot, C_rot (Bt,T,H,[R,]N), one row per head, dtype of B, and
    angle_final (Bt,H,K) fp32.  B, C are (Bt,T,G,N) or (Bt,T,G,R,N) with G
    dividing H; theta (Bt,T,H,K) gives H and the number K of rotated pairs."""
    if B.dim() == 4:
        Bt, T, G, N = B.shape
        R = 1
    else:
        Bt, T, G, R, N = B.shape
    H, K = theta.shape[2], theta.shape[3]
    if out is None:
        shape = (Bt, T, H, N) if B.dim() == 4 else (Bt, T, H, R, N)
        out = (torch.empty(shape, device=B.device, dtype=B.dtype),
               torch.empty(shape, device=B.device, dtype=B.dtype),
               torch.empty(Bt, H, K, device=B.device, dtype=torch.float32))
    Br, Cr, ang = out
    w, f, dev, io = "m3_rope_bc", torch.float32, B.device, _io_dtype("m3_rope_bc", B)
    _expect(w, dev, "C", C, B.numel(), io)
    _expect(w, dev, "theta", theta, Bt * T * H * K, f)
    _expect(w, dev, "dt", dt, Bt * T * H, f)
    _expect(w, dev, "angle0", angle0, Bt * H * K, f, required=False)
    _expect(w, dev, "B_rot", Br, Bt * T * H * R * N, io)
    _expect(w, dev, "C_rot", Cr, Bt * T * H * R * N, io)
    _expect(w, dev, "angle_final", ang, Bt * H * K, f, required=False)
    _expect_norm(w, dev, norm, H, R, N)
    nptr, keep = _norm(norm)
    d = Dims(Bt, T, H, 1, N, R, 1, G, K)
    _check(lib().m3_rope_bc(_ptr(B), _ptr(C), _DTYPE[B.dtype], _ptr(theta), _ptr(dt), _ptr(angle0),
                            nptr, d, _ptr(Br), _ptr(Cr), _ptr(ang), _stream(stream)), "m3_rope_bc")
    return Br, Cr, ang


def _state_outs(x, N, P, K, out):
    Bt, T, H = x.shape[0], x.shape[1], x.shape[2]
    if out is not None:
        return out
    dev = x.device
    return (torch.empty_like(x), torch.empty(Bt, H, N, P, device=dev, dtype=torch.float32),
            torch.empty(Bt, H, N, P, device=dev, dtype=torch.float32),
            torch.empty(Bt, H, K, device=dev, dtype=torch.float32))


def _expect_scan(w, x, dt, A, lam, theta, B, C, D, R, W_x=None, W_y=None, norm=None, h0=None, prevBx0=None,
                 angle0=None):
    """Element counts of the chunked scan's inputs: x (Bt,T,H,P); dt, lam
    (Bt,T,H); A, D (H); theta (Bt,T,H,K); B, C (Bt,T,G,[R,]N); W_x, W_y
    (H,R,P); h0, prevBx0 (Bt,H,N,P); angle0 (Bt,H,K)."""
    Bt, T, H, P = x.shape
    N, G, K = B.shape[-1], B.shape[2], theta.shape[-1]
    f, dev, io = torch.float32, x.device, _io_dtype(w, x)
    for name, t in (("dt", dt), ("lam", lam)):
        _expect(w, dev, name, t, Bt * T * H, f)
    for name, t in (("A", A), ("D", D)):
        _expect(w, dev, name, t, H, f)
    _expect(w, dev, "theta", theta, Bt * T * H * K, f)
    _expect(w, dev, "B", B, Bt * T * G * R * N, io)
    _expect(w, dev, "C", C, Bt * T * G * R * N, io)
    for name, t in (("W_x", W_x), ("W_y", W_y)):
        _expect(w, dev, name, t, H * R * P, f, required=False)
    for name, t in (("h0", h0), ("prevBx0", prevBx0)):
        _expect(w, dev, name, t, Bt * H * N * P, f, required=False)
    _expect(w, dev, "angle0", angle0, Bt * H * K, f, required=False)
    _expect_norm(w, dev, norm, H, R, N)
    return io


def _expect_state_outs(w, x, N, K, outs):
    Bt, T, H, P = x.shape
    y, hf, uf, af = outs
    f, dev = torch.float32, x.device
    _expect(w, dev, "y", y, x.numel(), x.dtype)
    _expect(w, dev, "h_final", hf, Bt * H * N * P, f, required=False)
    _expect(w, dev, "prevBx_final", uf, Bt * H * N * P, f, required=False)
    _expect(w, dev, "angle_final", af, Bt * H * K, f, required=False)


def _workspace(which, d, dtype, workspace, dev):
    need = workspace_bytes(which, d, dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None and workspace.device != dev:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return workspace, nbytes


def siso_chunked_fwd(x, dt, A, lam, theta, B, C, D, chunk, norm=None, h0=None, prevBx0=None,
                     angle0=None, workspace=None, out=None, stream=None):
    """S1+S2+S3: returns y (Bt,T,H,P), h_final, prevBx_final (Bt,H,N,P), angle_final
    (Bt,H,K).  B, C (Bt,T,G,N) with G dividing H; theta (Bt,T,H,K)."""
    Bt, T, H, P = x.shape
    N, G, K = B.shape[-1], B.shape[2], theta.shape[-1]
    w = "m3_siso_chunked_fwd"
    _expect_scan(w, x, dt, A, lam, theta, B, C, D, 1, norm=norm, h0=h0, prevBx0=prevBx0, angle0=angle0)
    y, hf, uf, af = _state_outs(x, N, P, K, out)
    _expect_state_outs(w, x, N, K, (y, hf, uf, af))
    d = Dims(Bt, T, H, P, N, 1, int(chunk), G, K)
    dtype = _DTYPE[x.dtype]
    ws, nbytes = _workspace(M3_WS_SISO, d, dtype, workspace, x.device)
    nptr, keep = _norm(norm)
    _check(lib().m3_siso_chunked_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B),
                                     _ptr(C), _ptr(D), dtype, nptr, _ptr(h0), _ptr(prevBx0),
                                     _ptr(angle0), d, _ptr(y), _ptr(hf), _ptr(uf), _ptr(af),
                                     _ptr(ws), nbytes, _stream(stream)), "m3_siso_chunked_fwd")
    return y, hf, uf, af


def mimo_chunked_fwd(x, dt, A, lam, theta, B, C, D, chunk, W_x=None, W_y=None, norm=None, h0=None,
                     prevBx0=None, angle0=None, workspace=None, out=None, stream=None):
    """S4: B, C (Bt,T,G,R,N); W_x, W_y (H,R,P) or None for ones."""
    Bt, T, H, P = x.shape
    R, N, G, K = B.shape[-2], B.shape[-1], B.shape[2], theta.shape[-1]
    w = "m3_mimo_chunked_fwd"
    _expect_scan(w, x, dt, A, lam, theta, B, C, D, R, W_x, W_y, norm, h0, prevBx0, angle0)
    y, hf, uf, af = _state_outs(x, N, P, K, out)
    _expect_state_outs(w, x, N, K, (y, hf, uf, af))
    d = Dims(Bt, T, H, P, N, R, int(chunk), G, K)
    dtype = _DTYPE[x.dtype]
    ws, nbytes = _workspace(M3_WS_MIMO, d, dtype, workspace, x.device)
    nptr, keep = _norm(norm)
    _check(lib().m3_mimo_chunked_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B),
                                     _ptr(C), _ptr(D), _ptr(W_x), _ptr(W_y), dtype, nptr, _ptr(h0),
                                     _ptr(prevBx0), _ptr(angle0), d, _ptr(y), _ptr(hf), _ptr(uf),
                                     _ptr(af), _ptr(ws), nbytes, _stream(stream)),
           "m3_mimo_chunked_fwd")
    return y, hf, uf, af


def _expect_decode(w, x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, R, y, h, angle, W_x=None, W_y=None,
                   norm=None):
    """Element counts of a decode step's arguments: x_t, y (Bt,H,P); dt_t,
    lam_t (Bt,H); A, D (H); theta_t, angle (Bt,H,K); B_t, C_t (Bt,G,[R,]N);
    W_x, W_y (H,R,P); h (Bt,H,N,P)."""
    Bt, H, P = x_t.shape
    N, G, K = B_t.shape[-1], B_t.shape[1], theta_t.shape[-1]
    f, dev, io = torch.float32, x_t.device, _io_dtype(w, x_t)
    for name, t in (("dt_t", dt_t), ("lam_t", lam_t)):
        _expect(w, dev, name, t, Bt * H, f)
    for name, t in (("A", A), ("D", D)):
        _expect(w, dev, name, t, H, f)
    _expect(w, dev, "theta_t", theta_t, Bt * H * K, f)
    _expect(w, dev, "B_t", B_t, Bt * G * R * N, io)
    _expect(w, dev, "C_t", C_t, Bt * G * R * N, io)
    for name, t in (("W_x", W_x), ("W_y", W_y)):
        _expect(w, dev, name, t, H * R * P, f, required=False)
    _expect(w, dev, "y_t", y, Bt * H * P, io)
    _expect(w, dev, "h", h, Bt * H * N * P, f)
    _expect(w, dev, "angle", angle, Bt * H * K, f)
    _expect_norm(w, dev, norm, H, R, N)


def step_decode(x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, h, prevBx, angle, norm=None, y_out=None,
                stream=None):
    """S5: one decode step; B_t, C_t (Bt,G,N); theta_t (Bt,H,K); h, prevBx, angle
    are updated in place; returns y_t (Bt,H,P)."""
    Bt, H, P = x_t.shape
    N, G, K = B_t.shape[-1], B_t.shape[1], theta_t.shape[-1]
    y = torch.empty_like(x_t) if y_out is None else y_out
    w = "m3_step_decode"
    _expect_decode(w, x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, 1, y, h, angle, norm=norm)
    _expect(w, x_t.device, "prevBx", prevBx, h.numel(), torch.float32)
    d = Dims(Bt, 1, H, P, N, 1, 1, G, K)
    nptr, keep = _norm(norm)
    _check(lib().m3_step_decode(_ptr(x_t), _ptr(dt_t), _ptr(A), _ptr(lam_t), _ptr(theta_t),
                                _ptr(B_t), _ptr(C_t), _ptr(D), _DTYPE[x_t.dtype], nptr, d, _ptr(h),
                                _ptr(prevBx), _ptr(angle), _ptr(y), _stream(stream)),
           "m3_step_decode")
    return y


def mimo_step_decode(x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, h, prevBx, angle, W_x=None, W_y=None,
                     norm=None, y_out=None, stream=None):
    """S5 for rank R: one decode step on the full previous-input state.  B_t, C_t
    (Bt,G,R,N); h, prevBx, angle updated in place; returns y_t (Bt,H,P)."""
    Bt, H, P = x_t.shape
    R, N, G, K = B_t.shape[-2], B_t.shape[-1], B_t.shape[1], theta_t.shape[-1]
    y = torch.empty_like(x_t) if y_out is None else y_out
    w = "m3_mimo_step_decode"
    _expect_decode(w, x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, R, y, h, angle, W_x, W_y, norm)
    _expect(w, x_t.device, "prevBx", prevBx, h.numel(), torch.float32)
    d = Dims(Bt, 1, H, P, N, R, 1, G, K)
    nptr, keep = _norm(norm)
    _check(lib().m3_mimo_step_decode(_ptr(x_t), _ptr(dt_t), _ptr(A), _ptr(lam_t), _ptr(theta_t), _ptr(B_t),
                                     _ptr(C_t), _ptr(D), _ptr(W_x), _ptr(W_y), _DTYPE[x_t.dtype], nptr, d,
                                     _ptr(h), _ptr(prevBx), _ptr(angle), _ptr(y), _stream(stream)),
           "m3_mimo_step_decode")
    return y


def step_decode_factored(x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, h, b_prev, x_prev, angle, W_x=None,
                         W_y=None, norm=None, y_out=None, stream=None):
    """One decode step on the factored previous-input state (any rank; B_t, C_t
    (Bt,G,R,N)).  h, b_prev (Bt,H,R,N), x_prev (Bt,H,P) and angle are updated in
    place; returns y_t (Bt,H,P)."""
    Bt, H, P = x_t.shape
    R, N, G, K = B_t.shape[-2], B_t.shape[-1], B_t.shape[1], theta_t.shape[-1]
    y = torch.empty_like(x_t) if y_out is None else y_out
    w = "m3_step_decode_factored"
    _expect_decode(w, x_t, dt_t, A, lam_t, theta_t, B_t, C_t, D, R, y, h, angle, W_x, W_y, norm)
    _expect(w, x_t.device, "b_prev", b_prev, Bt * H * R * N, torch.float32)
    _expect(w, x_t.device, "x_prev", x_prev, Bt * H * P, torch.float32)
    d = Dims(Bt, 1, H, P, N, R, 1, G, K)
    nptr, keep = _norm(norm)
    _check(lib().m3_step_decode_factored(_ptr(x_t), _ptr(dt_t), _ptr(A), _ptr(lam_t), _ptr(theta_t),
                                         _ptr(B_t), _ptr(C_t), _ptr(D), _ptr(W_x), _ptr(W_y),
                                         _DTYPE[x_t.dtype], nptr, d, _ptr(h), _ptr(b_prev), _ptr(x_prev),
                                         _ptr(angle), _ptr(y), _stream(stream)),
           "m3_step_decode_factored")
    return y


def chunked_bwd(x, dt, A, lam, theta, B, C, D, dy, chunk, W_x=None, W_y=None, norm=None, h0=None,
                prevBx0=None, angle0=None, dh_final=None, dprevBx_final=None, dangle_final=None,
                want=None, out=None, workspace=None, stream=None):
    """Backward of the chunked forward: returns a dict of fp32 gradients (the
    names in ``want``, by default all of them, without dW_x and dW_y for SISO;
    the gain and bias entries only when that part of the norm is on).  B, C
    (Bt,T,G,N) for SISO or (Bt,T,G,R,N) for rank R; dy has x's shape and dtype;
    the state adjoints default to zero.  ``out`` may hold preallocated fp32
    tensors by name (they are written and returned)."""
    Bt, T, H, P = x.shape
    R = B.shape[3] if B.dim() == 5 else 1
    N, G, K = B.shape[-1], B.shape[2], theta.shape[-1]
    mimo = B.dim() == 5
    w, f = "m3_chunked_bwd", torch.float32
    io = _expect_scan(w, x, dt, A, lam, theta, B, C, D, R, W_x, W_y, norm, h0, prevBx0, angle0)
    _expect(w, x.device, "dy", dy, x.numel(), io)
    for name, t, n in (("dh_final", dh_final, Bt * H * N * P), ("dprevBx_final", dprevBx_final, Bt * H * N * P),
                       ("dangle_final", dangle_final, Bt * H * K)):
        _expect(w, x.device, name, t, n, f, required=False)
    if want is None:
        want = tuple(k for k in GRAD_FIELDS if mimo or k not in ("dW_x", "dW_y"))
    dev = x.device
    shapes = dict(dx=x.shape, ddt=dt.shape, dA=A.shape, dlam=lam.shape, dtheta=theta.shape, dB=B.shape,
                  dC=C.shape, dD=D.shape, dW_x=(H, R, P), dW_y=(H, R, P), dnormw_B=(N,), dnormw_C=(N,),
                  dbias_B=(H, R, N), dbias_C=(H, R, N), dh0=(Bt, H, N, P), dprevBx0=(Bt, H, N, P),
                  dangle0=(Bt, H, K))
    nm = norm or {}
    off = {"dnormw_B": "normw_B", "dnormw_C": "normw_C", "dbias_B": "bias_B", "dbias_C": "bias_C"}
    pre = out or {}
    out = {k: (pre[k] if k in pre else torch.empty(shapes[k], device=dev, dtype=torch.float32)) for k in want
           if k not in off or nm.get(off[k]) is not None}
    for k, t in out.items():
        n = 1
        for e in shapes[k]:
            n *= e
        _expect(w, dev, k, t, n, f)
    g = Grads(*[_ptr(out.get(k)) for k in GRAD_FIELDS])
    d = Dims(Bt, T, H, P, N, R if mimo else 1, int(chunk), G, K)
    dtype = _DTYPE[x.dtype]
    ws, nbytes = _workspace(M3_WS_BWD_MIMO if mimo else M3_WS_BWD_SISO, d, dtype, workspace, dev)
    nptr, keep = _norm(norm)
    _check(lib().m3_chunked_bwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(B), _ptr(C), _ptr(D),
                                _ptr(W_x), _ptr(W_y), dtype, nptr, _ptr(h0), _ptr(prevBx0), _ptr(angle0), d,
                                _ptr(dy), _ptr(dh_final), _ptr(dprevBx_final), _ptr(dangle_final),
                                ctypes.byref(g), _ptr(ws), nbytes, _stream(stream)), "m3_chunked_bwd")
    return out


# ---- linear attention with a decay for each head, group norm -------------------
# These calls are short on the device (a single token's takes a few
# microseconds), so what only depends on the sizes is worked out once for each
# set of sizes: the dims structure and the workspace that the library asks for.
def _row_ptr(t):
    """Address of a tensor whose strides the caller has checked."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


# the current stream's handle without building a Stream object (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(fn, where, args, dev):
    """fn(*args, stream) on dev, which the library's launches need as the
    current device, and on its current stream."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(fn, where, args, dev)
    _check(fn(*args, torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(dev.index)),
           where)


def _on(stream, t, fn, *args, **kw):
    """fn on the caller's stream: as the current one, so that what the call
    allocates has no work of another stream pending on its memory; the
    caller's current stream is noted on the results, which it may read."""
    if stream.device != t.device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
    here = torch.cuda.current_stream(t.device)
    with torch.cuda.stream(stream):
        got = fn(*args, **kw)
    for r in (got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)):
        if r is not None:
            r.record_stream(here)
    return got


def _ld(where, name, t):
    """Elements between the rows of consecutive tokens of a (Bt,[T,]heads,d)
    tensor whose rows are contiguous: a slice of a fused projection has more
    than heads * d."""
    size = t.shape
    heads, d = size[-2], size[-1]
    ld = heads * d
    if t.is_contiguous():
        return ld
    stride = t.stride()
    ok = (d <= 1 or stride[-1] == 1) and (heads <= 1 or stride[-2] == d)
    if len(size) == 3:
        if size[0] > 1:
            ld = stride[0]
    else:
        B, T = size[:2]
        if T > 1:
            ld = stride[1]
            ok = ok and (B <= 1 or stride[0] == T * ld)
        elif B > 1:
            ld = stride[0]
    if not ok or ld < heads * d:
        raise ValueError("%s: %s has strides %s; the rows of a token have to be contiguous and the batch stride "
                         "seqlen times the token stride" % (where, name, tuple(stride)))
    return ld


@functools.lru_cache(maxsize=512)
def _linattn_plan(B, T, H, dv, dk, G, ldq, ldk, ldv, dtype, which):
    """The dims structure of a set of sizes, and its workspace (which: a query
    of m3_linattn_workspace_bytes, or None)."""
    d = LinattnDims(B, T, H, dv, dk, G, ldq, ldk, ldv)
    return d, (0 if which is None else int(lib().m3_linattn_workspace_bytes(which, d, dtype)))


def _linattn_dims(w, q, k, v, seq, which=None):
    vs, qs = v.shape, q.shape
    if len(qs) != 3 + seq or len(vs) != 3 + seq:
        raise ValueError("%s: q, k, v are (Bt,%sheads,d)" % (w, "T," if seq else ""))
    dt = _DTYPE.get(v.dtype)
    if dt is None:
        raise ValueError("%s: q, k, v must be float32 or bfloat16, got %s" % (w, v.dtype))
    dev, io = v.device, v.dtype
    if qs != k.shape or qs[:-2] != vs[:-2] or q.dtype != io or k.dtype != io or q.device != dev or k.device != dev:
        n = q.numel() // max(1, qs[-2] * qs[-1]) * qs[-2] * qs[-1]
        _expect(w, dev, "q", q, v.numel() // max(1, vs[-2] * vs[-1]) * qs[-2] * qs[-1], io)
        _expect(w, dev, "k", k, n, io)
        raise ValueError("%s: q is %s, k %s and v %s" % (w, tuple(qs), tuple(k.shape), tuple(vs)))
    H, G = vs[-2], qs[-2]
    if G < 1 or H % G or qs[-1] < 1:
        raise ValueError("%s: %d heads over %d groups of q and k, %d wide" % (w, H, G, qs[-1]))
    d, need = _linattn_plan(vs[0], vs[1] if seq else 1, H, vs[-1], qs[-1], G, _ld(w, "q", q), _ld(w, "k", k),
                            _ld(w, "v", v), dt, which)
    return d, need, dev, dt


def _like(t):
    """An output of t's shape and type, contiguous."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _own_workspace(need, workspace, t):
    dev = t.device
    if workspace is None:
        return (t.new_empty(need, dtype=torch.uint8) if need else None), need
    if workspace.device != dev:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
    return workspace, workspace.numel() * workspace.element_size()


def linattn_chunked_fwd(q, k, v, log_decay, scale=None, s0=None, lengths=None, workspace=None, out=None,
                        stream=None):
    """Linear attention with a decay for each head over a prompt:
    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t.

    q, k (Bt,T,G,dk) with G dividing H, v (Bt,T,H,dv), bf16 or fp32 (slices of
    a fused projection are taken as they are); log_decay (H) fp32, <= 0; scale
    defaults to dk^-1/2; s0 (Bt,H,dk,dv) fp32 or None for zero; lengths (Bt)
    int32 on the device or None: tokens behind a sequence's length are left
    out and their rows of y are zeros.  Returns y (Bt,T,H,dv) and s_final
    (Bt,H,dk,dv) fp32, the state for linattn_step_decode; ``out`` may hold
    both (s_final None when it is not wanted; like every output they must not
    overlap an input).  bf16 on the tensor cores: each term of y meets one
    rounding to bf16 before its fp32 sum; s_final does not (include/m3.h)."""
    if stream is not None:
        return _on(stream, v, linattn_chunked_fwd, q, k, v, log_decay, scale, s0, lengths, workspace, out)
    w, f = "m3_linattn_chunked_fwd", torch.float32
    d, need, dev, dt = _linattn_dims(w, q, k, v, True, M3_WS_LINATTN_FWD)
    ns = d.batch * d.nheads * d.dstate * d.headdim
    _expect(w, dev, "log_decay", log_decay, d.nheads, f)
    _expect(w, dev, "s0", s0, ns, f, required=False)
    _expect(w, dev, "lengths", lengths, d.batch, torch.int32, required=False)
    if out is None:
        y = _like(v)
        sf = v.new_empty((d.batch, d.nheads, d.dstate, d.headdim), dtype=f) if s0 is None else torch.empty_like(s0)
    else:
        y, sf = out
        _expect(w, dev, "y", y, v.numel(), v.dtype)
        _expect(w, dev, "s_final", sf, ns, f, required=False)
    ws, nbytes = _own_workspace(need, workspace, v)
    args = (_row_ptr(q), _row_ptr(k), _row_ptr(v), dt, _ptr(log_decay),
            d.dstate ** -0.5 if scale is None else float(scale), _ptr(s0), _ptr(lengths), d, _ptr(y), _ptr(sf),
            _ptr(ws), nbytes)
    _run(lib().m3_linattn_chunked_fwd, w, args, dev)
    return y, sf


def linattn_step_decode(q_t, k_t, v_t, log_decay, s, scale=None, y_out=None, stream=None):
    """One token of every lane: q_t, k_t (Bt,G,dk), v_t (Bt,H,dv); the state s
    (Bt,H,dk,dv) fp32 is updated in place; returns y_t (Bt,H,dv)."""
    if stream is not None:
        return _on(stream, v_t, linattn_step_decode, q_t, k_t, v_t, log_decay, s, scale, y_out)
    w, f = "m3_linattn_step_decode", torch.float32
    d, _, dev, dt = _linattn_dims(w, q_t, k_t, v_t, False)
    _expect(w, dev, "log_decay", log_decay, d.nheads, f)
    _expect(w, dev, "s", s, d.batch * d.nheads * d.dstate * d.headdim, f)
    if y_out is None:
        y = _like(v_t)
    else:
        y = y_out
        _expect(w, dev, "y_t", y, v_t.numel(), v_t.dtype)
    args = (_row_ptr(q_t), _row_ptr(k_t), _row_ptr(v_t), dt, _ptr(log_decay),
            d.dstate ** -0.5 if scale is None else float(scale), d, _ptr(s), _ptr(y))
    _run(lib().m3_linattn_step_decode, w, args, dev)
    return y


def linattn_chunked_bwd(q, k, v, log_decay, dy, scale=None, s0=None, ds_final=None, lengths=None, want=None,
                        out=None, workspace=None, stream=None):
    """Backward of linattn_chunked_fwd: a dict of the gradients named in
    ``want`` (by default dq, dk, dv, ds0), contiguous in their inputs' shapes
    and dtype (ds0 fp32).  dy (Bt,T,H,dv) contiguous; ds_final fp32 or None for
    zero.  ``out`` may hold preallocated tensors by name."""
    if stream is not None:
        return _on(stream, v, linattn_chunked_bwd, q, k, v, log_decay, dy, scale, s0, ds_final, lengths, want, out,
                   workspace)
    w, f = "m3_linattn_chunked_bwd", torch.float32
    d, need, dev, dt = _linattn_dims(w, q, k, v, True, M3_WS_LINATTN_BWD)
    ns = d.batch * d.nheads * d.dstate * d.headdim
    _expect(w, dev, "log_decay", log_decay, d.nheads, f)
    _expect(w, dev, "dy", dy, v.numel(), v.dtype)
    _expect(w, dev, "s0", s0, ns, f, required=False)
    _expect(w, dev, "ds_final", ds_final, ns, f, required=False)
    _expect(w, dev, "lengths", lengths, d.batch, torch.int32, required=False)
    names = ("dq", "dk", "dv", "ds0")
    shapes = dict(dq=q.shape, dk=k.shape, dv=v.shape, ds0=(d.batch, d.nheads, d.dstate, d.headdim))
    want = names if want is None else want
    pre = out or {}
    out = {}
    for n in want:
        if n not in shapes:
            raise ValueError("%s: no gradient %r" % (w, n))
        io = f if n == "ds0" else v.dtype
        if n in pre:
            out[n] = pre[n]
            _expect(w, dev, n, out[n], ns if n == "ds0" else {"dq": q, "dk": k, "dv": v}[n].numel(), io)
        else:
            out[n] = _like({"dq": q, "dk": k, "dv": v}[n]) if n != "ds0" else v.new_empty(shapes[n], dtype=io)
    ws, nbytes = _own_workspace(need, workspace, v)
    g = LinattnGrads(*[_ptr(out[n]) if n in out else None for n in names])
    args = (_row_ptr(q), _row_ptr(k), _row_ptr(v), dt, _ptr(log_decay),
            d.dstate ** -0.5 if scale is None else float(scale), _ptr(s0), _ptr(lengths), d, _ptr(dy), _ptr(ds_final),
            ctypes.byref(g), _ptr(ws), nbytes)
    _run(lib().m3_linattn_chunked_bwd, w, args, dev)
    return out


@functools.lru_cache(maxsize=512)
def _norm_plan(B, L, C, groups, dtype, which):
    d = NormDims(B, L, C, groups)
    return d, int(lib().m3_group_norm_workspace_bytes(which, d, dtype))


def _norm_dims(w, x, groups, weight, bias, gate, act, which):
    if x.dim() < 2:
        raise ValueError("%s: x is (Bt,...,C)" % w)
    if x.dtype not in _DTYPE:
        raise ValueError("%s: x must be float32 or bfloat16, got %s" % (w, x.dtype))
    if act not in ACTIVATIONS:
        raise ValueError("%s: act is one of %s, got %r" % (w, ", ".join(sorted(ACTIVATIONS)), act))
    C, B, dev = x.shape[-1], x.shape[0], x.device
    L = 1
    for n in x.shape[1:-1]:
        L *= n
    for name, t in (("weight", weight), ("bias", bias)):
        _expect(w, dev, name, t, C, torch.float32, required=False)
    _expect(w, dev, "gate", gate, x.numel(), x.dtype, required=False)
    dt = _DTYPE[x.dtype]
    return (*_norm_plan(B, L, C, int(groups), dt, which), dev, dt)


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5, workspace=None, out=None,
                   stream=None):
    """Group norm with an activation, channels last: u = (x - mean) rstd weight
    + bias with the statistics of each (x[b], group) over all positions and
    the group's channels; y = act(u), or u * act(gate) with a gate.

    x and gate (Bt,...,C) bf16 or fp32, contiguous; weight, bias (C) fp32 or
    None; act "none", "silu", "gelu" (erf) or "relu".  For the norm of each
    head of each token pass (tokens, C) and groups = heads.  Returns y, mean
    and rstd (Bt, groups) fp32, NaN where a sequence has no positions; ``out``
    may hold the three (mean, rstd None when not wanted)."""
    if stream is not None:
        return _on(stream, x, group_norm_fwd, x, groups, weight, bias, gate, act, eps, workspace, out)
    w, f = "m3_group_norm_fwd", torch.float32
    d, need, dev, dt = _norm_dims(w, x, groups, weight, bias, gate, act, M3_WS_NORM_FWD)
    if out is None:
        y, mean = _like(x), x.new_empty((d.batch, max(d.ngroups, 0)), dtype=f)
        rstd = torch.empty_like(mean)
    else:
        y, mean, rstd = out
        _expect(w, dev, "y", y, x.numel(), x.dtype)
        _expect(w, dev, "mean", mean, d.batch * d.ngroups, f, required=False)
        _expect(w, dev, "rstd", rstd, d.batch * d.ngroups, f, required=False)
    ws, nbytes = _own_workspace(need, workspace, x)
    args = (_ptr(x), dt, _ptr(weight), _ptr(bias), _ptr(gate), ACTIVATIONS[act], float(eps), d, _ptr(y), _ptr(mean),
            _ptr(rstd), _ptr(ws), nbytes)
    _run(lib().m3_group_norm_fwd, w, args, dev)
    if d.seqlen == 0:                                     # the library writes nothing then
        for t in (mean, rstd):
            if t is not None:
                t.fill_(float("nan"))
    return y, mean, rstd


def group_norm_bwd(x, dy, mean, rstd, groups, weight=None, bias=None, gate=None, act="none", want=None, out=None,
                   workspace=None, stream=None):
    """Backward of group_norm_fwd from its mean and rstd: a dict of the
    gradients named in ``want`` (by default dx, dweight, dbias, and dgate with
    a gate): dx, dgate in x's shape and dtype, dweight, dbias (C) fp32."""
    if stream is not None:
        return _on(stream, x, group_norm_bwd, x, dy, mean, rstd, groups, weight, bias, gate, act, want, out, workspace)
    w, f = "m3_group_norm_bwd", torch.float32
    d, need, dev, dt = _norm_dims(w, x, groups, weight, bias, gate, act, M3_WS_NORM_BWD)
    _expect(w, dev, "dy", dy, x.numel(), x.dtype)
    _expect(w, dev, "mean", mean, d.batch * d.ngroups, f)
    _expect(w, dev, "rstd", rstd, d.batch * d.ngroups, f)
    names = ("dx", "dweight", "dbias", "dgate")
    if want is None:
        want = names if gate is not None else names[:3]
    pre = out or {}
    out = {}
    for n in want:
        if n not in names or (n == "dgate" and gate is None):
            raise ValueError("%s: no gradient %r" % (w, n))
        wide = n in ("dx", "dgate")
        shape, io = (x.shape, x.dtype) if wide else ((d.channels,), f)
        if n in pre:
            out[n] = pre[n]
            _expect(w, dev, n, out[n], x.numel() if wide else d.channels, io)
        else:
            of = x if wide else weight if n == "dweight" else bias
            out[n] = x.new_empty(shape, dtype=io) if of is None else _like(of)
    ws, nbytes = _own_workspace(need, workspace, x)
    args = (_ptr(x), _ptr(dy), dt, _ptr(weight), _ptr(bias), _ptr(gate), ACTIVATIONS[act], _ptr(mean), _ptr(rstd), d,
            _ptr(out.get("dx")), _ptr(out.get("dweight")), _ptr(out.get("dbias")), _ptr(out.get("dgate")), _ptr(ws),
            nbytes)
    _run(lib().m3_group_norm_bwd, w, args, dev)
    return out
