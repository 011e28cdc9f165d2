"""B200 selective scan (S6): Python binding of libssmscan.so.

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream; every step of the scan runs in the library's CUDA
kernels (include/ssm_scan.h).  There is no CPU path.

    y, last_state = scan_fwd(u, delta, A, B, C, D, z, delta_bias,
                             delta_softplus=True, return_last_state=True)
    grads = scan_bwd(u, delta, A, B, C, D, z, delta_bias, dout)
    y_t = scan_step(u_t, delta_t, A, B_t, C_t, D, z_t, delta_bias, state=state)

    y, last = gated_scan_fwd(u, f, z, f_bias, return_last_state=True)
    grads = gated_scan_bwd(u, f, z, f_bias, dout)
    y_t = gated_scan_step(u_t, f_t, z_t, f_bias, state=state)
    y, residual = layer_norm(x, weight, bias, residual=residual)
    grads = layer_norm_bwd(residual, weight, bias, dy, dresidual_out=dresidual)

Layouts: u, delta, z, y, dout (batch, dim, seqlen); B, C (batch, seqlen,
dstate); A (dim, dstate) fp32; D, delta_bias (dim,) fp32; states (batch, dim,
dstate) fp32.  io tensors are all bf16 or all fp32.
"""
from __future__ import annotations

import ctypes
import functools

from . import _lib
from ._lib import (PATH_NAMES, SSM_BF16, SSM_F32, SSM_FLAG_SAVE_STATES,  # noqa: F401
                   SSM_FLAG_TOKEN_MAJOR, SSM_FLAG_UNTIED, SSM_FLAG_ZOH_EXACT, SSM_PATH_AUTO,
                   SSM_PATH_LOOKBACK, SSM_PATH_LOOKBACK_WS, SSM_PATH_PER_GROUP, SSM_PATH_SPLIT_L,
                   ssm_shape)

__all__ = ["scan_fwd", "scan_bwd", "scan_step", "causal_conv1d", "causal_conv1d_bwd", "fwd_workspace_bytes", "bwd_workspace_bytes",
           "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "gated_scan_shape", "gated_scan_path",
           "gated_scan_fwd_workspace_bytes", "gated_scan_bwd_workspace_bytes", "layer_norm", "layer_norm_bwd",
           "layer_norm_bwd_workspace_bytes", "fwd_path", "check", "ScanError", "make_shape"]


class ScanError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_lib.status_string(code)} ({code})")
        self.code = code


def _io_dtype(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError(f"io tensors must be bfloat16 or float32, got {t.dtype}")


def make_shape(batch: int, dim: int, seqlen: int, dstate: int, io_dtype: int,
               path: int = SSM_PATH_AUTO, lanes: int = 0, flags: int = 0) -> ssm_shape:
    return ssm_shape(batch, dim, seqlen, dstate, io_dtype, path, lanes, flags)


def fwd_workspace_bytes(shape: ssm_shape) -> int:
    return int(_lib.load().ssm_scan_fwd_workspace_bytes(ctypes.byref(shape)))


def bwd_workspace_bytes(shape: ssm_shape) -> int:
    return int(_lib.load().ssm_scan_bwd_workspace_bytes(ctypes.byref(shape)))


def fwd_path(shape: ssm_shape) -> str:
    return PATH_NAMES[int(_lib.load().ssm_scan_fwd_path(ctypes.byref(shape)))]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_io(name, t, shape, dtype, device):
    if t is None:
        return
    # one combined test on the common path; the message is built only on failure
    if t.is_cuda and t.device == device and t.shape == tuple(shape) and t.dtype == dtype and t.is_contiguous():
        return
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _workspace(nbytes, device, workspace):
    import torch
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace holds {workspace.nbytes} bytes, needs {nbytes}")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, delta_softplus=True,
             initial_state=None, y=None, last_state=None, return_last_state=False,
             workspace=None, path: int = SSM_PATH_AUTO, lanes: int = 0, zoh_exact=False,
             save_states=False, token_major=False, check_status=False, stream=None):
    """Forward selective scan; returns y, or (y, last_state).  zoh_exact selects the
    exact zero-order-hold input term instead of the Euler one (Delta * B).
    save_states also writes the state entering every 8-step chunk into
    ``workspace`` (which must then be given), for scan_bwd(fwd_workspace=...).
    token_major: u, delta, z and y are (batch, seqlen, dim) instead.
    The look-back schedules hand states between warps with a bounded wait that
    records a give-up in the workspace's error word instead of trapping:
    check_status=True synchronises after the launch and raises ScanError
    (SSM_ERR_DEVICE_TIMEOUT) if that happened; otherwise pass a workspace and
    call check(workspace) when convenient (an internal workspace is not kept)."""
    import torch
    if token_major:
        batch, seqlen, dim = u.shape
    else:
        batch, dim, seqlen = u.shape
    dstate = B.shape[-1]
    dt = u.dtype
    dev = u.device
    f32 = torch.float32
    act = (batch, seqlen, dim) if token_major else (batch, dim, seqlen)
    _check_io("u", u, act, dt, dev)
    _check_io("delta", delta, act, dt, dev)
    _check_io("z", z, act, dt, dev)
    _check_io("B", B, (batch, seqlen, dstate), dt, dev)
    _check_io("C", C, (batch, seqlen, dstate), dt, dev)
    _check_io("A", A, (dim, dstate), f32, dev)
    _check_io("D", D, (dim,), f32, dev)
    _check_io("delta_bias", delta_bias, (dim,), f32, dev)
    _check_io("initial_state", initial_state, (batch, dim, dstate), f32, dev)
    if y is None:
        y = torch.empty_like(u)
    _check_io("y", y, act, dt, dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, dim, dstate), dtype=f32, device=dev)
    _check_io("last_state", last_state, (batch, dim, dstate), f32, dev)
    flags = ((SSM_FLAG_ZOH_EXACT if zoh_exact else 0) | (SSM_FLAG_SAVE_STATES if save_states else 0)
             | (SSM_FLAG_TOKEN_MAJOR if token_major else 0))
    if save_states and workspace is None:
        raise ValueError("save_states writes into the workspace: pass workspace=")
    shape = make_shape(batch, dim, seqlen, dstate, _io_dtype(u), path, lanes, flags)
    nbytes = fwd_workspace_bytes(shape)
    if nbytes == 0 and batch * dim * seqlen > 0:
        raise ScanError(_lib.SSM_ERR_UNSUPPORTED, "ssm_scan_fwd_workspace_bytes")
    ws = _workspace(nbytes, dev, workspace)
    rc = _lib.load().ssm_scan_fwd(
        ctypes.byref(shape), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
        _ptr(delta_bias), int(bool(delta_softplus)), _ptr(initial_state), _ptr(y),
        _ptr(last_state), _ptr(ws), ctypes.c_size_t(ws.numel()), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_scan_fwd")
    if check_status:
        check(ws, stream)
    if return_last_state:
        return y, last_state
    return y


@functools.lru_cache(maxsize=64)
def _step_shape(batch, dim, dstate, io_dtype, flags):
    # read-only for the library (a const pointer): one struct per shape serves
    # every decode step of that shape
    return make_shape(batch, dim, 1, dstate, io_dtype, flags=flags)


def scan_step(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, state,
              delta_softplus=True, zoh_exact=False, y=None, stream=None):
    """One recurrent step for every (batch, channel): updates `state` in place
    and returns y.  u, delta, z, y (batch, dim); B, C (batch, dstate); state
    (batch, dim, dstate) fp32."""
    import torch
    batch, dim = u.shape
    dstate = B.shape[-1]
    dt = u.dtype
    dev = u.device
    f32 = torch.float32
    _check_io("u", u, (batch, dim), dt, dev)
    _check_io("delta", delta, (batch, dim), dt, dev)
    _check_io("z", z, (batch, dim), dt, dev)
    _check_io("B", B, (batch, dstate), dt, dev)
    _check_io("C", C, (batch, dstate), dt, dev)
    _check_io("A", A, (dim, dstate), f32, dev)
    _check_io("D", D, (dim,), f32, dev)
    _check_io("delta_bias", delta_bias, (dim,), f32, dev)
    _check_io("state", state, (batch, dim, dstate), f32, dev)
    if y is None:
        y = torch.empty_like(u)
    _check_io("y", y, (batch, dim), dt, dev)
    shape = _step_shape(batch, dim, dstate, _io_dtype(u), SSM_FLAG_ZOH_EXACT if zoh_exact else 0)
    rc = _lib.load().ssm_scan_step(
        ctypes.byref(shape), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
        _ptr(delta_bias), int(bool(delta_softplus)), _ptr(state), _ptr(y), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_scan_step")
    return y


def causal_conv1d(x, weight, bias=None, *, initial_state=None, silu=True, out=None,
                  return_final_state=False, final_state=None, stream=None):
    """Causal depthwise conv1d along seqlen (+ SiLU); x, out (batch, dim, seqlen),
    weight (dim, width) fp32, states (batch, dim, width - 1) fp32."""
    import torch
    batch, dim, seqlen = x.shape
    width = weight.shape[-1]
    dev = x.device
    f32 = torch.float32
    _check_io("x", x, (batch, dim, seqlen), x.dtype, dev)
    _check_io("weight", weight, (dim, width), f32, dev)
    _check_io("bias", bias, (dim,), f32, dev)
    _check_io("initial_state", initial_state, (batch, dim, width - 1), f32, dev)
    if out is None:
        out = torch.empty_like(x)
    _check_io("out", out, (batch, dim, seqlen), x.dtype, dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, dim, width - 1), dtype=f32, device=dev)
    _check_io("final_state", final_state, (batch, dim, width - 1), f32, dev)
    rc = _lib.load().ssm_causal_conv1d(
        batch, dim, seqlen, width, _io_dtype(x), _ptr(x), _ptr(weight), _ptr(bias),
        _ptr(initial_state), int(bool(silu)), _ptr(out), _ptr(final_state), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_causal_conv1d")
    if return_final_state:
        return out, final_state
    return out


def causal_conv1d_bwd(x, weight, bias, dout, *, initial_state=None, silu=True,
                      want_dinitial_state=False, stream=None):
    """Backward of causal_conv1d: returns dict(dx, dweight, dbias, dinitial_state)."""
    import torch
    batch, dim, seqlen = x.shape
    width = weight.shape[-1]
    dev, f32 = x.device, torch.float32
    _check_io("x", x, (batch, dim, seqlen), x.dtype, dev)
    _check_io("dout", dout, (batch, dim, seqlen), x.dtype, dev)
    _check_io("weight", weight, (dim, width), f32, dev)
    _check_io("bias", bias, (dim,), f32, dev)
    _check_io("initial_state", initial_state, (batch, dim, width - 1), f32, dev)
    g = {"dx": torch.empty_like(x), "dweight": torch.empty((dim, width), dtype=f32, device=dev),
         "dbias": torch.empty((dim,), dtype=f32, device=dev) if bias is not None else None,
         "dinitial_state": (torch.empty((batch, dim, width - 1), dtype=f32, device=dev)
                            if want_dinitial_state else None)}
    rc = _lib.load().ssm_causal_conv1d_bwd(
        batch, dim, seqlen, width, _io_dtype(x), _ptr(x), _ptr(weight), _ptr(bias),
        _ptr(initial_state), int(bool(silu)), _ptr(dout), _ptr(g["dx"]), _ptr(g["dweight"]),
        _ptr(g["dbias"]), _ptr(g["dinitial_state"]), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_causal_conv1d_bwd")
    return g


def scan_bwd(u, delta, A, B, C, D, z, delta_bias, dout, *, delta_softplus=True,
             initial_state=None, want_dinitial_state=False, out=None, workspace=None,
             fwd_workspace=None, zoh_exact=False, token_major=False, stream=None):
    """Backward of scan_fwd by recomputation; returns a dict of gradients.
    fwd_workspace: the workspace of a scan_fwd(save_states=True) call on the same
    inputs, whose saved chunk states the backward then uses.  zoh_exact: the
    exact zero-order-hold input term.  token_major: u, delta, z, dout and the
    du, ddelta, dz gradients are (batch, seqlen, dim)."""
    import torch
    if token_major:
        batch, seqlen, dim = u.shape
    else:
        batch, dim, seqlen = u.shape
    dstate = B.shape[-1]
    dt, dev, f32 = u.dtype, u.device, torch.float32
    act = (batch, seqlen, dim) if token_major else (batch, dim, seqlen)
    for name, t, shp, ty in (("u", u, act, dt), ("delta", delta, act, dt),
                             ("z", z, act, dt), ("B", B, (batch, seqlen, dstate), dt),
                             ("C", C, (batch, seqlen, dstate), dt), ("A", A, (dim, dstate), f32),
                             ("D", D, (dim,), f32), ("delta_bias", delta_bias, (dim,), f32),
                             ("dout", dout, act, dt),
                             ("initial_state", initial_state, (batch, dim, dstate), f32)):
        _check_io(name, t, shp, ty, dev)
    g = dict(out or {})
    g.setdefault("du", torch.empty_like(u))
    g.setdefault("ddelta", torch.empty_like(u))
    g.setdefault("dA", torch.empty((dim, dstate), dtype=f32, device=dev))
    g.setdefault("dB", torch.empty_like(B))
    g.setdefault("dC", torch.empty_like(C))
    g.setdefault("dD", torch.empty((dim,), dtype=f32, device=dev) if D is not None else None)
    g.setdefault("dz", torch.empty_like(u) if z is not None else None)
    g.setdefault("ddelta_bias",
                 torch.empty((dim,), dtype=f32, device=dev) if delta_bias is not None else None)
    g.setdefault("dinitial_state",
                 torch.empty((batch, dim, dstate), dtype=f32, device=dev) if want_dinitial_state else None)
    flags = ((SSM_FLAG_SAVE_STATES if fwd_workspace is not None else 0)
             | (SSM_FLAG_ZOH_EXACT if zoh_exact else 0) | (SSM_FLAG_TOKEN_MAJOR if token_major else 0))
    shape = make_shape(batch, dim, seqlen, dstate, _io_dtype(u), flags=flags)
    nbytes = bwd_workspace_bytes(shape)
    ws = _workspace(nbytes, dev, workspace)
    rc = _lib.load().ssm_scan_bwd(
        ctypes.byref(shape), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
        _ptr(delta_bias), int(bool(delta_softplus)), _ptr(initial_state), _ptr(dout),
        _ptr(fwd_workspace), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
        _ptr(g["dD"]), _ptr(g["dz"]), _ptr(g["ddelta_bias"]), _ptr(g["dinitial_state"]),
        _ptr(ws), ctypes.c_size_t(ws.numel()), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_scan_bwd")
    return g


# ---- gated linear recurrence and layer norm ------------------------------------
# The host's share of a call decides the smallest ones (a decode step's kernel takes 2 us),
# so the common path is kept short: one combined test per tensor, addresses passed as plain
# integers, the stream's handle without a Stream object.
class _launch:
    """``with _launch(device, stream) as handle:`` makes the caller's stream, or the tensors'
    own device, current for a launch; what the call allocates belongs to that stream."""
    __slots__ = ("device", "stream", "guard")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        import torch
        if self.stream is None:
            self.guard = torch.cuda.device(self.device)
        else:
            if self.stream.device != self.device:
                raise ValueError(f"stream is on {self.stream.device}, the tensors on {self.device}")
            self.guard = torch.cuda.stream(self.stream)
        self.guard.__enter__()
        s = self.stream if self.stream is not None else torch.cuda.current_stream(self.device)
        return s.cuda_stream

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)


_raw_stream = None


def _on_stream(device, stream, call):
    """call(handle) with the launch's stream and device current."""
    global _raw_stream
    import torch
    if stream is None and torch.cuda.current_device() == device.index:
        if _raw_stream is None:
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda index: torch.cuda.current_stream(index).cuda_stream)
        return call(_raw_stream(device.index))
    with _launch(device, stream) as handle:
        return call(handle)


def _fits(t, shape, dtype, index):
    # index: the CUDA device's (a CPU tensor has -1)
    return t is None or (t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous())


def _addr(t):
    return None if t is None else t.data_ptr()


def _cuda_device(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _workspace_for(nbytes, device, workspace):
    """A caller's workspace checked, or a new one; None where none is needed."""
    import torch
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    if not workspace.is_cuda or workspace.device != device:
        raise ValueError(f"workspace must be on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.nbytes < nbytes:
        raise ValueError(f"workspace holds {workspace.nbytes} bytes, needs {nbytes}")
    return workspace


@functools.lru_cache(maxsize=256)
def _gated_shape(batch, dim, seqlen, io_dtype, path, flags):
    # read-only for the library (a const pointer): one struct serves every call of a shape, and
    # so never leaves the binding (gated_scan_shape makes the caller's)
    return make_shape(batch, dim, seqlen, 1, io_dtype, path, flags=flags)


@functools.lru_cache(maxsize=256)
def _gated_step_ref(batch, dim, io_dtype, flags):
    return ctypes.byref(_gated_shape(batch, dim, 1, io_dtype, SSM_PATH_AUTO, flags))


def _gated_key(u, tied, save_states, token_major, path):
    if u.dim() != 3:
        raise ValueError(f"u has shape {tuple(u.shape)}, expected three axes")
    batch, dim, seqlen = u.shape
    flags = 0 if tied else SSM_FLAG_UNTIED
    if save_states:
        flags |= SSM_FLAG_SAVE_STATES
    if token_major:
        flags |= SSM_FLAG_TOKEN_MAJOR
        dim, seqlen = seqlen, dim
    return batch, dim, seqlen, _io_dtype(u), path, flags


@functools.lru_cache(maxsize=256)
def _gated_plan(key, device_index):
    """(shape, reference to it, forward and backward workspace bytes on the device)."""
    import torch
    shape = _gated_shape(*key)
    with torch.cuda.device(device_index):
        return (shape, ctypes.byref(shape), gated_scan_fwd_workspace_bytes(shape),
                gated_scan_bwd_workspace_bytes(shape))


def gated_scan_shape(u, *, tied=True, save_states=False, token_major=False, path: int = SSM_PATH_AUTO) -> ssm_shape:
    """The shape of a gated_scan_fwd / gated_scan_bwd call on ``u``, for the workspace queries:
    a struct of the caller's own."""
    batch, dim, seqlen, io_dtype, path, flags = _gated_key(u, tied, save_states, token_major, path)
    return make_shape(batch, dim, seqlen, 1, io_dtype, path, flags=flags)


def gated_scan_fwd_workspace_bytes(shape: ssm_shape) -> int:
    return int(_lib.load().ssm_gated_scan_fwd_workspace_bytes(ctypes.byref(shape)))


def gated_scan_bwd_workspace_bytes(shape: ssm_shape) -> int:
    return int(_lib.load().ssm_gated_scan_bwd_workspace_bytes(ctypes.byref(shape)))


def gated_scan_path(shape: ssm_shape) -> str:
    return PATH_NAMES[int(_lib.load().ssm_gated_scan_path(ctypes.byref(shape)))]


def _check_starts(starts, batch, seqlen, dev):
    import torch
    if starts is None:
        return None
    if starts.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"starts has dtype {starts.dtype}, expected bool or uint8")
    _check_io("starts", starts, (batch, seqlen), starts.dtype, dev)
    return starts


def _check_gated(shape, u, f, z, f_bias, starts, initial_state):
    import torch
    batch, dim, dt, dev, f32 = shape.batch, shape.dim, u.dtype, u.device, torch.float32
    act, per, states, at = u.shape, (dim,), (batch, dim), u.get_device()
    if (starts is None and u.is_contiguous() and _fits(f, act, dt, at) and _fits(z, act, dt, at)
            and _fits(f_bias, per, f32, at) and _fits(initial_state, states, f32, at)):
        return
    _check_io("u", u, act, dt, dev)
    _check_io("f", f, act, dt, dev)
    _check_io("z", z, act, dt, dev)
    _check_io("f_bias", f_bias, per, f32, dev)
    _check_io("initial_state", initial_state, states, f32, dev)
    _check_starts(starts, batch, shape.seqlen, dev)


def gated_scan_fwd(u, f, z=None, f_bias=None, *, tied=True, starts=None, initial_state=None, y=None,
                   last_state=None, return_last_state=False, workspace=None, path: int = SSM_PATH_AUTO,
                   save_states=False, token_major=False, check_status=False, stream=None):
    """Gated linear recurrence over whole sequences; returns y, or (y, last_state).

    With a_t = sigmoid(f_t + f_bias): h_t = a_t h_{t-1} + (1 - a_t) u_t (``tied``) or
    h_t = a_t h_{t-1} + u_t (``tied=False``: u is gated already), y_t = h_t SiLU(z_t).
    u, f, z, y (batch, dim, seqlen), or (batch, seqlen, dim) with token_major; f_bias
    (dim,) and the states (batch, dim) fp32.  starts (batch, seqlen), bool or uint8: a
    packed sequence starts there, so h_{t-1} counts as 0 (initial_state too, at t = 0).
    save_states writes the states gated_scan_bwd(fwd_workspace=...) needs into
    ``workspace`` (which must then be given).  check_status: as in scan_fwd.  The call runs
    on the tensors' device, on ``stream`` or that device's current one."""
    import torch
    dev = _cuda_device("u", u)
    shape, ref, nbytes, _ = _gated_plan(_gated_key(u, tied, save_states, token_major, path), dev.index)
    _check_gated(shape, u, f, z, f_bias, starts, initial_state)
    if save_states and workspace is None:
        raise ValueError("save_states writes into the workspace: pass workspace=")
    states = (shape.batch, shape.dim)
    if y is not None:
        _check_io("y", y, u.shape, u.dtype, dev)
    if last_state is not None:
        _check_io("last_state", last_state, states, torch.float32, dev)
    lib = _lib.load()

    def call(handle):
        out = torch.empty_like(u) if y is None else y
        last = last_state
        if last is None and return_last_state:
            last = u.new_empty(states, dtype=torch.float32)
        ws = None if workspace is None and nbytes == 0 else _workspace_for(nbytes, dev, workspace)
        rc = lib.ssm_gated_scan_fwd(ref, u.data_ptr(), f.data_ptr(), _addr(z), _addr(f_bias), _addr(starts),
                                    _addr(initial_state), out.data_ptr(), _addr(last), _addr(ws),
                                    0 if ws is None else ws.nbytes, handle)
        if rc != 0:
            raise ScanError(rc, "ssm_gated_scan_fwd")
        if check_status and nbytes:
            check(ws, stream)
        return (out, last) if return_last_state else out

    return _on_stream(dev, stream, call)


def gated_scan_bwd(u, f, z, f_bias, dout, *, tied=True, starts=None, initial_state=None, dlast_state=None,
                   want_dinitial_state=False, out=None, workspace=None, fwd_workspace=None,
                   path: int = SSM_PATH_AUTO, token_major=False, check_status=False, stream=None):
    """Backward of gated_scan_fwd by recomputation; returns a dict of the gradients
    du, df, dz, df_bias, dinitial_state (None for what is absent).  dlast_state
    (batch, dim) fp32: the gradient reaching last_state.  fwd_workspace: the workspace
    of a gated_scan_fwd(save_states=True) call on the same inputs, with the same ``path``."""
    import torch
    dev = _cuda_device("u", u)
    shape, ref, fwd_bytes, nbytes = _gated_plan(
        _gated_key(u, tied, fwd_workspace is not None, token_major, path), dev.index)
    _check_gated(shape, u, f, z, f_bias, starts, initial_state)
    f32, states, per = torch.float32, (shape.batch, shape.dim), (shape.dim,)
    _check_io("dout", dout, u.shape, u.dtype, dev)
    _check_io("dlast_state", dlast_state, states, f32, dev)
    lib = _lib.load()
    given = out or {}
    if fwd_workspace is not None:
        _workspace_for(fwd_bytes, dev, fwd_workspace)

    def gradient(name, like, shp, ty):
        if given.get(name) is not None:
            _check_io(name, given[name], shp, ty, dev)
            return given[name]
        return None if like is None else u.new_empty(shp, dtype=ty)

    def call(handle):
        g = {"du": gradient("du", u, u.shape, u.dtype), "df": gradient("df", u, u.shape, u.dtype),
             "dz": gradient("dz", z, u.shape, u.dtype), "df_bias": gradient("df_bias", f_bias, per, f32),
             "dinitial_state": gradient("dinitial_state", u if want_dinitial_state else None, states, f32)}
        ws = _workspace_for(nbytes, dev, workspace)
        rc = lib.ssm_gated_scan_bwd(
            ref, u.data_ptr(), f.data_ptr(), _addr(z), _addr(f_bias), _addr(starts), _addr(initial_state),
            dout.data_ptr(), _addr(dlast_state), _addr(fwd_workspace), g["du"].data_ptr(), g["df"].data_ptr(),
            _addr(g["dz"]), _addr(g["df_bias"]), _addr(g["dinitial_state"]), _addr(ws),
            0 if ws is None else ws.nbytes, handle)
        if rc != 0:
            raise ScanError(rc, "ssm_gated_scan_bwd")
        if check_status and ws is not None:
            check(ws, stream)
        return g

    return _on_stream(dev, stream, call)


def gated_scan_step(u, f, z=None, f_bias=None, *, state, tied=True, y=None, stream=None):
    """One token of the gated recurrence for every (batch, channel): updates ``state``
    (batch, dim) fp32 in place and returns y.  u, f, z, y (batch, dim)."""
    import torch
    dev = _cuda_device("u", u)
    act, dt, f32, at = u.shape, u.dtype, torch.float32, u.get_device()
    batch, dim = act
    if not (u.is_contiguous() and _fits(f, act, dt, at) and _fits(z, act, dt, at) and _fits(y, act, dt, at)
            and _fits(f_bias, (dim,), f32, at) and _fits(state, act, f32, at)):
        for name, t, shp, ty in (("u", u, act, dt), ("f", f, act, dt), ("z", z, act, dt), ("y", y, act, dt),
                                 ("f_bias", f_bias, (dim,), f32), ("state", state, act, f32)):
            _check_io(name, t, shp, ty, dev)
    ref = _gated_step_ref(batch, dim, _io_dtype(u), 0 if tied else SSM_FLAG_UNTIED)

    def call(handle):
        out = torch.empty_like(u) if y is None else y
        rc = _lib.load().ssm_gated_scan_step(ref, u.data_ptr(), f.data_ptr(), _addr(z), _addr(f_bias),
                                             state.data_ptr(), out.data_ptr(), handle)
        if rc != 0:
            raise ScanError(rc, "ssm_gated_scan_step")
        return out

    return _on_stream(dev, stream, call)


def _residual_dtype(name, t, io) -> int:
    import torch
    if t.dtype != io and t.dtype != torch.float32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {io} or {torch.float32}")
    return _io_dtype(t)


def layer_norm(x, weight, bias=None, *, residual=None, eps=1e-5, y=None, residual_out=None, stream=None):
    """Layer norm over the last axis, with the residual stream's addition before it.

    Without ``residual`` returns y = norm(x) * weight + bias.  With it returns (y, s):
    s = x + residual, rounded to the residual's dtype (x's or fp32), and y = norm(s) *
    weight + bias.  x, y (..., dim) bf16 or fp32; weight, bias (dim,) fp32.
    residual_out may be residual itself."""
    import torch
    dev = _cuda_device("x", x)
    if x.dim() < 1:
        raise ValueError("x needs at least one axis")
    act, dt, f32 = x.shape, x.dtype, torch.float32
    dim = act[-1]
    rows = x.numel() // dim if dim else 0
    io = rd = _io_dtype(x)
    rt = dt
    if residual is not None:
        rd, rt = _residual_dtype("residual", residual, dt), residual.dtype
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    at = x.get_device()
    if not (x.is_contiguous() and _fits(weight, (dim,), f32, at) and _fits(bias, (dim,), f32, at)
            and _fits(residual, act, rt, at) and _fits(y, act, dt, at) and _fits(residual_out, act, rt, at)):
        for name, t, shp, ty in (("x", x, act, dt), ("weight", weight, (dim,), f32), ("bias", bias, (dim,), f32),
                                 ("residual", residual, act, rt), ("y", y, act, dt),
                                 ("residual_out", residual_out, act, rt)):
            _check_io(name, t, shp, ty, dev)

    def call(handle):
        out = torch.empty_like(x) if y is None else y
        total = residual_out
        if total is None and residual is not None:
            total = torch.empty_like(residual)
        rc = _lib.load().ssm_layer_norm(rows, dim, io, rd, x.data_ptr(), _addr(residual), weight.data_ptr(),
                                        _addr(bias), eps, out.data_ptr(), _addr(total), handle)
        if rc != 0:
            raise ScanError(rc, "ssm_layer_norm")
        return out if residual is None else (out, total)

    return _on_stream(dev, stream, call)


def layer_norm_bwd_workspace_bytes(rows: int, dim: int) -> int:
    return int(_lib.load().ssm_layer_norm_bwd_workspace_bytes(rows, dim))


def layer_norm_bwd(s, weight, bias, dy, *, eps=1e-5, dresidual_out=None, out=None, workspace=None, stream=None):
    """Backward of layer_norm; returns dict(dx, dresidual, dweight, dbias).

    s: what was normalised (layer_norm's second result, or x where there was no
    residual), whose dtype is dy's or fp32; dresidual_out: the gradient reaching s past
    the norm, in s's dtype.  dx has dy's dtype; dresidual is the gradient of the
    residual in s's dtype, the same tensor as dx where the two dtypes are one.  bias:
    the forward's, or None for no dbias."""
    import torch
    dev = _cuda_device("dy", dy)
    if dy.dim() < 1:
        raise ValueError("dy needs at least one axis")
    act, dt, f32 = dy.shape, dy.dtype, torch.float32
    dim = act[-1]
    rows = dy.numel() // dim if dim else 0
    io, rd, rt = _io_dtype(dy), _residual_dtype("s", s, dt), s.dtype
    for name, t, shp, ty in (("s", s, act, rt), ("dy", dy, act, dt), ("weight", weight, (dim,), f32),
                             ("bias", bias, (dim,), f32), ("dresidual_out", dresidual_out, act, rt)):
        _check_io(name, t, shp, ty, dev)
    lib = _lib.load()
    given = out or {}
    for name, wanted in (("dresidual", io != rd), ("dbias", bias is not None)):
        if not wanted and given.get(name) is not None:
            raise ValueError(f"out holds {name}, which this call has no use for")

    def gradient(name, wanted, shp, ty):
        if wanted and given.get(name) is not None:
            _check_io(name, given[name], shp, ty, dev)
            return given[name]
        return torch.empty(shp, dtype=ty, device=dev) if wanted else None

    def call(handle):
        g = {"dx": gradient("dx", True, act, dt), "dresidual": gradient("dresidual", io != rd, act, rt),
             "dweight": gradient("dweight", True, (dim,), f32), "dbias": gradient("dbias", bias is not None, (dim,), f32)}
        ws = _workspace_for(lib.ssm_layer_norm_bwd_workspace_bytes(rows, dim), dev, workspace)
        rc = lib.ssm_layer_norm_bwd(rows, dim, io, rd, s.data_ptr(), weight.data_ptr(), eps, dy.data_ptr(),
                                    _addr(dresidual_out), g["dx"].data_ptr(), _addr(g["dresidual"]),
                                    g["dweight"].data_ptr(), _addr(g["dbias"]), _addr(ws),
                                    0 if ws is None else ws.nbytes, handle)
        if rc != 0:
            raise ScanError(rc, "ssm_layer_norm_bwd")
        if io == rd:
            g["dresidual"] = g["dx"]
        return g

    return _on_stream(dev, stream, call)


def check(workspace, stream=None) -> None:
    """Synchronise and raise ScanError if a device-side wait gave up."""
    rc = _lib.load().ssm_scan_check(_ptr(workspace), _stream(stream))
    if rc != 0:
        raise ScanError(rc, "ssm_scan_check")
