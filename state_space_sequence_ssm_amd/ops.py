"""Thin torch binding of the C ABI: its entry points by the same names,
marshalling device tensors into the argument structures.  Every step of the
computation runs in the HIP kernels of libm3ssm.so; torch only provides device
memory and the current stream (and copies a token's rows that lie too far apart
for the library, in m3_selective_scan_step).

Nothing here is recorded for automatic differentiation: outputs carry no gradient
history, also where inputs require gradients.  Gradients come from the `_backward`
entry points; a torch.autograd.Function around a pair of them records both.
"""
from __future__ import annotations

import ctypes
import functools
import inspect

import torch

from . import _lib


class M3Error(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {_lib.status_string(code)} ({code})")
        self.code = code


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.M3_BF16
    if t.dtype == torch.float32:
        return _lib.M3_F32
    raise TypeError(f"unsupported input dtype {t.dtype}; use bfloat16 or float32")


def _ptr(t, dtype=None, shape=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _prologue(pro, H, R, N, bc_norm, bc_eps, B_norm_w, C_norm_w, B_bias, C_bias, dt_softplus, dt_bias):
    """Fill the m3_prologue of an argument structure (steps fused in front of
    the core: B / C RMS normalisation, head biases, Delta = softplus)."""
    f32 = torch.float32
    pro.bc_norm = 1 if bc_norm else 0
    pro.dt_softplus = 1 if dt_softplus else 0
    pro.bc_eps = float(bc_eps)
    pro.B_norm_w = _ptr(B_norm_w, f32, (N,), "B_norm_w")
    pro.C_norm_w = _ptr(C_norm_w, f32, (N,), "C_norm_w")
    pro.B_bias = _ptr(B_bias, f32, (H, R, N), "B_bias")
    pro.C_bias = _ptr(C_bias, f32, (H, R, N), "C_bias")
    pro.dt_bias = _ptr(dt_bias, f32, (H,), "dt_bias")


def m3_ssm_prefill(x, B, C, dt, lam, A, theta=None, h0=None, Bprev_rot=None, xprev=None, phi0=None,
                   *, y=None, h_final=None, Bprev_rot_out=None, xprev_out=None, phi_out=None,
                   want_state=True, want_carry=False, chunk=0, workspace=None, omega=None, A_tok=None,
                   head_major=False, noalloc=False, bc_norm=False, bc_eps=1e-6, B_norm_w=None, C_norm_w=None,
                   B_bias=None, C_bias=None, dt_softplus=False, dt_bias=None, stream=None):
    """Chunked prefill.  Shapes: x [Bt,L,H,R,P], B/C [Bt,L,H,R,N] (bf16 or fp32),
    dt/lam [Bt,L,H] fp32, A [H] fp32, theta [Bt,L,H,N/2] fp32 or None (or
    instead omega [Bt,L,N/2] fp32: rates shared by the heads, theta = dt * omega
    formed on chip); A_tok [Bt,L,H] fp32: A per token (then
    A may be None); optional
    carry-in h0 [Bt,H,N,P], Bprev_rot [Bt,H,R,N], xprev [Bt,H,R,P], phi0 [Bt,H,N/2].
    Output tensors are allocated when not given.  workspace: a uint8 device
    tensor of at least prefill_workspace_bytes(...) bytes, None to allocate one
    when the library asks for it, or False to run without (unsplit).  Returns
    a dict with y and, as requested, h_final and the carry-out (Bprev_rot,
    xprev, phi).  head_major: x, B, C and y are [Bt,H,L,R,.] instead.
    noalloc: call m3_ssm_prefill_noalloc (the library's static scratch in
    place of a workspace; workspace must then be None).
    Prologue (computed on chip; B, C and dt are then the raw projections):
    bc_norm / bc_eps / B_norm_w, C_norm_w [N]: RMS normalisation of each B and
    C row; B_bias, C_bias [H,R,N]: head biases added after it; dt_softplus /
    dt_bias [H]: Delta = softplus(dt + dt_bias)."""
    if head_major:
        Bt, H, L, R, P = x.shape
    else:
        Bt, L, H, R, P = x.shape
    N = B.shape[-1]
    big = (lambda D: (Bt, H, L, R, D)) if head_major else (lambda D: (Bt, L, H, R, D))
    f32 = torch.float32
    if y is None:
        y = torch.empty_like(x)
    if want_state and h_final is None:
        h_final = torch.empty((Bt, H, N, P), device=x.device, dtype=f32)
    if want_carry:
        if Bprev_rot_out is None:
            Bprev_rot_out = torch.empty((Bt, H, R, N), device=x.device, dtype=f32)
        if xprev_out is None:
            xprev_out = torch.empty((Bt, H, R, P), device=x.device, dtype=x.dtype)
        if (theta is not None or omega is not None) and phi_out is None:
            phi_out = torch.empty((Bt, H, N // 2), device=x.device, dtype=f32)
    a = _lib.PrefillArgs()
    a.Bt, a.L, a.H, a.P, a.N, a.R, a.chunk = Bt, L, H, P, N, R, chunk
    a.in_dtype = _dtype_code(x)
    a.layout = 1 if head_major else 0
    a.x = _ptr(x, x.dtype, big(P), "x")
    a.B = _ptr(B, x.dtype, big(N), "B")
    a.C = _ptr(C, x.dtype, big(N), "C")
    a.dt = _ptr(dt, f32, (Bt, L, H), "dt")
    a.lam = _ptr(lam, f32, (Bt, L, H), "lam")
    a.A = _ptr(A, f32, (H,), "A")
    a.A_tok = _ptr(A_tok, f32, (Bt, L, H), "A_tok")
    a.theta = _ptr(theta, f32, (Bt, L, H, N // 2), "theta")
    a.omega = _ptr(omega, f32, (Bt, L, N // 2), "omega")
    a.h0 = _ptr(h0, f32, (Bt, H, N, P), "h0")
    a.Bprev_rot = _ptr(Bprev_rot, f32, (Bt, H, R, N), "Bprev_rot")
    a.xprev = _ptr(xprev, x.dtype, (Bt, H, R, P), "xprev")
    a.phi0 = _ptr(phi0, f32, (Bt, H, N // 2), "phi0")
    a.y = _ptr(y, x.dtype, big(P), "y")
    a.h_final = _ptr(h_final, f32, (Bt, H, N, P), "h_final")
    a.Bprev_rot_out = _ptr(Bprev_rot_out, f32, (Bt, H, R, N), "Bprev_rot_out")
    a.xprev_out = _ptr(xprev_out, x.dtype, (Bt, H, R, P), "xprev_out")
    a.phi_out = _ptr(phi_out, f32, (Bt, H, N // 2), "phi_out")
    _prologue(a.pro, H, R, N, bc_norm, bc_eps, B_norm_w, C_norm_w, B_bias, C_bias, dt_softplus, dt_bias)
    lib = _lib.load()
    if noalloc:
        if workspace is not None:
            raise ValueError("noalloc takes no workspace")
        rc = lib.m3_ssm_prefill_noalloc(ctypes.byref(a), _stream(stream))
        if rc != _lib.M3_OK:
            raise M3Error(rc, "m3_ssm_prefill_noalloc")
        return dict(y=y, h=h_final, Bprev_rot=Bprev_rot_out, xprev=xprev_out, phi=phi_out)
    if workspace is not False:
        need = lib.m3_ssm_prefill_workspace_size(ctypes.byref(a))
        if need > 0:
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
            a.workspace = _ptr(workspace, torch.uint8, None, "workspace")
            a.workspace_bytes = workspace.numel()
    rc = lib.m3_ssm_prefill(ctypes.byref(a), _stream(stream))
    if rc != _lib.M3_OK:
        raise M3Error(rc, "m3_ssm_prefill")
    return dict(y=y, h=h_final, Bprev_rot=Bprev_rot_out, xprev=xprev_out, phi=phi_out)


def m3_ssm_prefill_backward(x, B, C, dt, lam, A, theta=None, h0=None, Bprev_rot=None, xprev=None, phi0=None,
                            *, dy, dh_final=None, A_tok=None, want_carry_grads=False, workspace=None,
                            out=None, stream=None):
    """Gradients of the prefill for upstream dy [Bt,L,H,R,P] (bf16) and
    dh_final [Bt,H,N,P] (fp32, optional).  Forward inputs as for
    m3_ssm_prefill (bf16, token-major).  Returns a dict with dx, dB, dC (bf16),
    ddt, dlam (fp32 [Bt,L,H]), dA ([H], or [Bt,L,H] with A_tok), dtheta (with
    theta) and, with want_carry_grads, dh0, dBprev_rot, dxprev, dphi0.  `out`:
    optional dict of preallocated gradient tensors (any subset of those keys)."""
    Bt, L, H, R, P = x.shape
    N = B.shape[-1]
    f32, dev = torch.float32, x.device
    given = out
    out = dict(dx=torch.empty_like(x), dB=torch.empty_like(B), dC=torch.empty_like(C),
               ddt=torch.empty((Bt, L, H), device=dev, dtype=f32), dlam=torch.empty((Bt, L, H), device=dev, dtype=f32),
               dA=torch.empty((Bt, L, H) if A_tok is not None else (H,), device=dev, dtype=f32),
               dtheta=None if theta is None else torch.empty_like(theta),
               dh0=None, dBprev_rot=None, dxprev=None, dphi0=None)
    if want_carry_grads:
        out["dh0"] = torch.empty((Bt, H, N, P), device=dev, dtype=f32)
        if Bprev_rot is not None:
            out["dBprev_rot"] = torch.empty((Bt, H, R, N), device=dev, dtype=f32)
            out["dxprev"] = torch.empty((Bt, H, R, P), device=dev, dtype=x.dtype)
        if theta is not None:
            out["dphi0"] = torch.empty((Bt, H, N // 2), device=dev, dtype=f32)
    for k, v in (given or {}).items():
        out[k] = v
    a = _lib.BackwardArgs()
    a.Bt, a.L, a.H, a.P, a.N, a.R = Bt, L, H, P, N, R
    a.in_dtype = _dtype_code(x)
    big = lambda D: (Bt, L, H, R, D)  # noqa: E731
    a.x = _ptr(x, x.dtype, big(P), "x")
    a.B = _ptr(B, x.dtype, big(N), "B")
    a.C = _ptr(C, x.dtype, big(N), "C")
    a.dt = _ptr(dt, f32, (Bt, L, H), "dt")
    a.lam = _ptr(lam, f32, (Bt, L, H), "lam")
    a.A = _ptr(A, f32, (H,), "A")
    a.A_tok = _ptr(A_tok, f32, (Bt, L, H), "A_tok")
    a.theta = _ptr(theta, f32, (Bt, L, H, N // 2), "theta")
    a.h0 = _ptr(h0, f32, (Bt, H, N, P), "h0")
    a.Bprev_rot = _ptr(Bprev_rot, f32, (Bt, H, R, N), "Bprev_rot")
    a.xprev = _ptr(xprev, x.dtype, (Bt, H, R, P), "xprev")
    a.phi0 = _ptr(phi0, f32, (Bt, H, N // 2), "phi0")
    a.dy = _ptr(dy, x.dtype, big(P), "dy")
    a.dh_final = _ptr(dh_final, f32, (Bt, H, N, P), "dh_final")
    shapes = dict(dx=big(P), dB=big(N), dC=big(N), ddt=(Bt, L, H), dlam=(Bt, L, H),
                  dA=(Bt, L, H) if A_tok is not None else (H,), dtheta=(Bt, L, H, N // 2), dh0=(Bt, H, N, P),
                  dBprev_rot=(Bt, H, R, N), dxprev=(Bt, H, R, P), dphi0=(Bt, H, N // 2))
    for k in ("dx", "dB", "dC", "dxprev"):
        setattr(a, k, _ptr(out[k], x.dtype, shapes[k], k))
    for k in ("ddt", "dlam", "dA", "dtheta", "dh0", "dBprev_rot", "dphi0"):
        setattr(a, k, _ptr(out[k], f32, shapes[k], k))
    lib = _lib.load()
    need = lib.m3_ssm_prefill_backward_workspace_size(ctypes.byref(a))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    a.workspace = _ptr(workspace, torch.uint8, None, "workspace")
    a.workspace_bytes = workspace.numel()
    rc = lib.m3_ssm_prefill_backward(ctypes.byref(a), _stream(stream))
    if rc != _lib.M3_OK:
        raise M3Error(rc, "m3_ssm_prefill_backward")
    return out


def backward_workspace_bytes(Bt, L, H, P, N, R, rope=False):
    """Bytes of the workspace m3_ssm_prefill_backward needs for this shape."""
    a = _lib.BackwardArgs()
    a.Bt, a.L, a.H, a.P, a.N, a.R = Bt, L, H, P, N, R
    a.theta = 1 if rope else None  # only NULL-ness is read
    return _lib.load().m3_ssm_prefill_backward_workspace_size(ctypes.byref(a))


def prefill_workspace_bytes(Bt, L, H, P, N, R, dtype=torch.bfloat16, rope=False):
    """Bytes of the optional prefill workspace for this shape (0: none used)."""
    a = _lib.PrefillArgs()
    a.Bt, a.L, a.H, a.P, a.N, a.R = Bt, L, H, P, N, R
    a.in_dtype = _lib.M3_BF16 if dtype == torch.bfloat16 else _lib.M3_F32
    a.theta = 1 if rope else None  # only NULL-ness is read
    return _lib.load().m3_ssm_prefill_workspace_size(ctypes.byref(a))


def m3_ssm_decode_step(h, phi, Bprev_rot, xprev, x, B, C, dt, lam, A, theta=None, *, y=None, A_tok=None,
                       omega=None, bc_norm=False, bc_eps=1e-6, B_norm_w=None, C_norm_w=None, B_bias=None,
                       C_bias=None, dt_softplus=False, dt_bias=None, stream=None):
    """One decode token.  In/out (updated in place): h [Bt,H,N,P] fp32,
    phi [Bt,H,N/2] fp32 (None iff theta None), Bprev_rot [Bt,H,R,N] fp32,
    xprev [Bt,H,R,P].  Inputs x [Bt,H,R,P], B/C [Bt,H,R,N], dt/lam [Bt,H],
    A [H] (or A_tok [Bt,H]: this token's A; then A may be None), theta
    [Bt,H,N/2] or None (or omega [Bt,N/2]: rates shared by the heads, theta =
    dt * omega).  The prologue arguments are those of m3_ssm_prefill.
    Returns y [Bt,H,R,P]."""
    Bt, H, R, P = x.shape
    N = B.shape[-1]
    f32 = torch.float32
    if y is None:
        y = torch.empty_like(x)
    a = _lib.DecodeArgs()
    a.Bt, a.H, a.P, a.N, a.R = Bt, H, P, N, R
    a.in_dtype = _dtype_code(x)
    a.h = _ptr(h, f32, (Bt, H, N, P), "h")
    a.phi = _ptr(phi, f32, (Bt, H, N // 2), "phi")
    a.Bprev_rot = _ptr(Bprev_rot, f32, (Bt, H, R, N), "Bprev_rot")
    a.xprev = _ptr(xprev, x.dtype, (Bt, H, R, P), "xprev")
    a.x = _ptr(x, x.dtype, (Bt, H, R, P), "x")
    a.B = _ptr(B, x.dtype, (Bt, H, R, N), "B")
    a.C = _ptr(C, x.dtype, (Bt, H, R, N), "C")
    a.dt = _ptr(dt, f32, (Bt, H), "dt")
    a.lam = _ptr(lam, f32, (Bt, H), "lam")
    a.A = _ptr(A, f32, (H,), "A")
    a.A_tok = _ptr(A_tok, f32, (Bt, H), "A_tok")
    a.theta = _ptr(theta, f32, (Bt, H, N // 2), "theta")
    a.omega = _ptr(omega, f32, (Bt, N // 2), "omega")
    a.y = _ptr(y, x.dtype, (Bt, H, R, P), "y")
    _prologue(a.pro, H, R, N, bc_norm, bc_eps, B_norm_w, C_norm_w, B_bias, C_bias, dt_softplus, dt_bias)
    rc = _lib.load().m3_ssm_decode_step(ctypes.byref(a), _stream(stream))
    if rc != _lib.M3_OK:
        raise M3Error(rc, "m3_ssm_decode_step")
    return y


def m3_rope_angles_cumsum(theta, phi0=None, *, phi=None, stream=None):
    """Inclusive cumulative angles phi = phi0 + cumsum(theta, dim=1).
    theta [Bt,L,H,J] fp32; phi0 [Bt,H,J] or None.  Returns phi [Bt,L,H,J]."""
    Bt, L, H, J = theta.shape
    if phi is None:
        phi = torch.empty_like(theta)
    pt = _ptr(theta, torch.float32, (Bt, L, H, J), "theta")
    pp = _ptr(phi0, torch.float32, (Bt, H, J), "phi0")
    po = _ptr(phi, torch.float32, (Bt, L, H, J), "phi")
    rc = _lib.load().m3_rope_angles_cumsum(pt, pp, po, Bt, L, H, J, _stream(stream))
    if rc != _lib.M3_OK:
        raise M3Error(rc, "m3_rope_angles_cumsum")
    return phi


# ---------------------------------------------------------------- layer operators
def _scoped(fn):
    """Run a call on its first tensor's device and on `stream`: outputs and
    workspaces are then allocated for that stream as well."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        index = first.get_device()
        if index < 0:
            raise ValueError(f"{name} must be a device tensor")
        if stream is None and index == torch.cuda.current_device():
            return fn(*args, **kw)
        if stream is None:
            stream = torch.cuda.current_stream(first.device)
        elif stream.device != first.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


_MAX = (1 << 31) - 1


def _too_large(*v):
    """Refuse sizes of which the structures' 32-bit fields would keep the rest."""
    raise ValueError(f"sizes up to {_MAX} are taken, got {max(v)}")


def _refuse(t, dtype, shape, name, dev):
    """Say what is wrong with a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _dense(t, dtype, shape, name, dev):
    """Address of a dense tensor (None: NULL) on device index `dev` after checking it."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, dtype, shape, name, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, shape, lead, name, dev):
    """Address of a tensor whose first `lead` axes count rows, and the elements
    from one of its rows to the next: dense rows, the same distance apart
    throughout (0: dense)."""
    if t is None:
        return None, 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, dtype, shape, name, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0
    strides = t.stride()
    # the usual slices first (one or two axes of rows, one or two inside a row): 0.5 us
    # instead of 2, for up to five tensors of a call
    n, ld = len(shape), strides[lead - 1]
    if strides[-1] == 1 and shape[lead - 1] > 1 and (
            (n == lead + 1 and ld >= shape[-1]) or
            (n == lead + 2 and strides[lead] == shape[-1] and ld >= shape[-2] * shape[-1])) and (
            lead == 1 or (lead == 2 and strides[0] == ld * shape[1])):
        return t.data_ptr(), ld
    width = 1
    for n, st in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        if n > 1 and st != width:
            raise ValueError(f"{name}: the elements of a row must be dense")
        width *= n
    ld, rows = 0, 1
    for n, st in zip(reversed(shape[:lead]), reversed(strides[:lead])):
        if n == 1:
            continue
        if ld == 0:
            ld = st
            if st < width:
                raise ValueError(f"{name}: rows must not overlap")
        elif st != ld * rows:
            raise ValueError(f"{name}: all rows must be the same distance apart")
        rows *= n
    return t.data_ptr(), ld


def _out(given, dtype, shape, name, like, dev):
    """An output and its address: the given tensor after checking it, or a new one on
    the device of `like` (an input that is checked itself).  `like` is the input of the
    same shape and type where there is one: the fastest pattern, 1.2 us instead of 2.2."""
    if given is not None:
        return given, _dense(given, dtype, shape, name, dev)
    if dtype is like.dtype and like.shape == shape:
        given = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        given = torch.empty(shape, dtype=dtype, device=like.device)
    return given, given.data_ptr()


# The current stream's handle without building a Stream object, which takes as
# long as a launch (2.8 us of 13 for a single token's convolution).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_calls = {}


def _call_of(name):
    call = _calls.get(name)
    if call is None:
        call = _calls[name] = getattr(_lib.load(), name)
    return call


def _run_layer(name, args, dev):
    rc = _call_of(name)(ctypes.byref(args), _raw_stream(dev))
    if rc != _lib.M3_OK:
        raise M3Error(rc, name)


def _take_workspace(name, args, given, dev):
    """Put a workspace of the size the library asks for into the arguments: the
    given uint8 tensor, or a new one.  Returns it (it must outlive the call)."""
    need = _call_of(name + "_workspace_size")(ctypes.byref(args))
    if given is None:
        if need != 0:
            given = torch.empty(need, dtype=torch.uint8, device=dev)
            args.workspace, args.workspace_bytes = given.data_ptr(), need
        return given
    args.workspace = _dense(given, torch.uint8, given.shape, "workspace", dev)
    args.workspace_bytes = given.numel()
    return given


_F32 = torch.float32


@_scoped
def m3_causal_conv(x, w, bias=None, state=None, *, lengths=None, silu=True, y=None, state_out=None, want_state=False):
    """Short causal depthwise convolution over the tokens:
    y[t, d] = act(bias[d] + sum_k w[d, k] x[t - (W - 1) + k, d]), act = SiLU or
    identity.  x [Bt, L, D] (bf16 or fp32; rows may be slices of wider ones), w
    [D, W] fp32, W in 2..4, bias [D] fp32; state [Bt, W-1, D]: the inputs before
    the first token (None: zeros); lengths [Bt] int32: tokens held per item.
    Returns a dict with y [Bt, L, D] (rows behind an item's length are left as
    they were) and, with want_state or state_out (may be `state`), state: the
    last W - 1 inputs.  `stream`: the stream to run on (default: the current
    one), for this and the following operators.  No operator records its
    call for automatic differentiation: gradients come from `_backward`."""
    Bt, L, D = x.shape
    W = w.shape[-1]
    dev, t = x.get_device(), x.dtype
    a = _lib.ConvArgs()
    if Bt > _MAX or L > _MAX or D > _MAX or W > _MAX:
        _too_large(Bt, L, D, W)
    a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu = Bt, L, D, W, _dtype_code(x), 1 if silu else 0
    a.x, a.x_ld = _rows(x, t, x.shape, 2, "x", dev)
    a.w = _dense(w, _F32, (D, W), "w", dev)
    a.bias = _dense(bias, _F32, (D,), "bias", dev)
    a.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    a.state = _dense(state, t, (Bt, W - 1, D), "state", dev)
    y, a.y = _out(y, t, (Bt, L, D), "y", x, dev)
    if want_state or state_out is not None:
        state_out, a.state_out = _out(state_out, t, (Bt, W - 1, D), "state_out", x if state is None else state, dev)
    _run_layer("m3_causal_conv", a, dev)
    return dict(y=y, state=state_out)


@_scoped
def m3_causal_conv_step(state, x, w, bias=None, *, silu=True, y=None, state_out=None):
    """One token of m3_causal_conv: x [Bt, D], state [Bt, W-1, D] updated in
    place (or read only, the new one going to state_out).  Returns y [Bt, D]."""
    Bt, D = x.shape
    W = w.shape[-1]
    dev, t = state.get_device(), x.dtype
    a = _lib.ConvStepArgs()
    if Bt > _MAX or D > _MAX or W > _MAX:
        _too_large(Bt, D, W)
    a.Bt, a.D, a.W, a.in_dtype, a.silu = Bt, D, W, _dtype_code(x), 1 if silu else 0
    a.x, a.x_ld = _rows(x, t, x.shape, 1, "x", dev)
    a.w = _dense(w, _F32, (D, W), "w", dev)
    a.bias = _dense(bias, _F32, (D,), "bias", dev)
    a.state = _dense(state, t, (Bt, W - 1, D), "state", dev)
    a.state_out = _dense(state_out, t, (Bt, W - 1, D), "state_out", dev)
    y, a.y = _out(y, t, (Bt, D), "y", x, dev)
    _run_layer("m3_causal_conv_step", a, dev)
    return y


@_scoped
def m3_causal_conv_backward(x, w, bias=None, state=None, *, dy, lengths=None, silu=True, want_state_grad=False,
                            workspace=None, out=None):
    """Gradients of m3_causal_conv for dy [Bt, L, D] (dense).  Returns a dict
    with dx, dw [D, W], dbias [D] (None without bias) and, with
    want_state_grad, dstate.  `out`: optional dict of preallocated tensors."""
    Bt, L, D = x.shape
    W = w.shape[-1]
    dev, t = x.get_device(), x.dtype
    got = out or {}
    a = _lib.ConvBackwardArgs()
    if Bt > _MAX or L > _MAX or D > _MAX or W > _MAX:
        _too_large(Bt, L, D, W)
    a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu = Bt, L, D, W, _dtype_code(x), 1 if silu else 0
    a.x, a.x_ld = _rows(x, t, x.shape, 2, "x", dev)
    a.w = _dense(w, _F32, (D, W), "w", dev)
    a.bias = _dense(bias, _F32, (D,), "bias", dev)
    a.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    a.state = _dense(state, t, (Bt, W - 1, D), "state", dev)
    a.dy = _dense(dy, t, (Bt, L, D), "dy", dev)
    out = dict(dx=None, dw=None, dbias=None, dstate=None)
    out["dx"], a.dx = _out(got.get("dx"), t, (Bt, L, D), "dx", x, dev)
    out["dw"], a.dw = _out(got.get("dw"), _F32, (D, W), "dw", w, dev)
    if bias is not None:
        out["dbias"], a.dbias = _out(got.get("dbias"), _F32, (D,), "dbias", bias, dev)
    if want_state_grad or "dstate" in got:
        out["dstate"], a.dstate = _out(got.get("dstate"), t, (Bt, W - 1, D), "dstate", x if state is None else state, dev)
    workspace = _take_workspace("m3_causal_conv_backward", a, workspace, dev)
    _run_layer("m3_causal_conv_backward", a, dev)
    return out


# The library's limit of the scan's row distances.  A token's rows that lie further apart
# (one position of a batch of long sequences) are copied: they are small beside the state.
_FAR_ROWS = 1 << 24


def _scan_inputs(a, dev, lead, x, dt, A, B, C, D, z, dt_softplus, dt_bias):
    """The inputs that the scan, its backward and its step share."""
    G, N = B.shape[-2:]
    t, shape = x.dtype, x.shape
    width, n, bc = shape[-1], len(lead), (*lead, G, N)
    if width > _MAX or N > _MAX or G > _MAX or max(lead) > _MAX:
        _too_large(width, N, G, *lead)
    a.D, a.N, a.G, a.in_dtype, a.dt_softplus = width, N, G, _dtype_code(x), 1 if dt_softplus else 0
    a.x, a.x_ld = _rows(x, t, shape, n, "x", dev)
    a.dt, a.dt_ld = _rows(dt, t, shape, n, "dt", dev)
    a.z, a.z_ld = _rows(z, t, shape, n, "z", dev)
    a.B, a.B_ld = _rows(B, t, bc, n, "B", dev)
    a.C, a.C_ld = _rows(C, t, bc, n, "C", dev)
    a.A = _dense(A, _F32, (width, N), "A", dev)
    a.D_skip = _dense(D, _F32, (width,), "D", dev)
    a.dt_bias = _dense(dt_bias, _F32, (width,), "dt_bias", dev)


@_scoped
def m3_selective_scan(x, dt, A, B, C, D=None, z=None, h0=None, *, lengths=None, dt_softplus=False, dt_bias=None, y=None,
                      h_final=None, want_state=True, workspace=None):
    """Selective scan with a diagonal state per channel:
    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t . h_t + D x_t)
    silu(z_t), delta = softplus(dt + dt_bias) or dt itself.  x, dt, z
    [Bt, L, D], B, C [Bt, L, G, N] (bf16 or fp32; rows may be slices of wider
    ones); A [D, N], D [D], dt_bias [D], h0 [Bt, D, N] fp32; lengths [Bt] int32;
    N in 1..64.  workspace: a uint8 device tensor, None to allocate one when the
    library asks for it, or False to run without (token axis not cut).
    Returns a dict with y [Bt, L, D] (rows behind an item's length are left as
    they were) and h: the last state [Bt, D, N]."""
    Bt, L, width = x.shape
    N = A.shape[-1]
    dev = x.get_device()
    a = _lib.ScanArgs()
    a.Bt, a.L = Bt, L
    _scan_inputs(a, dev, (Bt, L), x, dt, A, B, C, D, z, dt_softplus, dt_bias)
    a.h0 = _dense(h0, _F32, (Bt, width, N), "h0", dev)
    a.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    y, a.y = _out(y, x.dtype, (Bt, L, width), "y", x, dev)
    if want_state or h_final is not None:
        h_final, a.h_final = _out(h_final, _F32, (Bt, width, N), "h_final", x if h0 is None else h0, dev)
    if workspace is not False:
        workspace = _take_workspace("m3_selective_scan", a, workspace, dev)
    _run_layer("m3_selective_scan", a, dev)
    return dict(y=y, h=h_final)


@_scoped
def m3_selective_scan_step(h, x, dt, A, B, C, D=None, z=None, *, dt_softplus=False, dt_bias=None, y=None, h_out=None):
    """One token of m3_selective_scan: x, dt, z [Bt, D], B, C [Bt, G, N], h
    [Bt, D, N] fp32 updated in place (or read only, the new state going to
    h_out).  Rows 2^24 elements apart and more are copied first.  Returns y
    [Bt, D]."""
    Bt, width = x.shape
    N = A.shape[-1]
    dev = h.get_device()
    a = _lib.ScanStepArgs()
    a.Bt = Bt
    _scan_inputs(a, dev, (Bt,), x, dt, A, B, C, D, z, dt_softplus, dt_bias)
    a.h = _dense(h, _F32, (Bt, width, N), "h", dev)
    a.h_out = _dense(h_out, _F32, (Bt, width, N), "h_out", dev)
    y, a.y = _out(y, x.dtype, (Bt, width), "y", x, dev)
    try:
        _run_layer("m3_selective_scan_step", a, dev)
    except M3Error:  # refused, and nothing launched: checked here, where it costs other calls nothing
        if max(a.x_ld, a.dt_ld, a.z_ld, a.B_ld, a.C_ld) < _FAR_ROWS:
            raise
        x, dt, z, B, C = (None if t is None else t.contiguous() for t in (x, dt, z, B, C))
        _scan_inputs(a, dev, (Bt,), x, dt, A, B, C, D, z, dt_softplus, dt_bias)
        _run_layer("m3_selective_scan_step", a, dev)
    return y


@_scoped
def m3_selective_scan_backward(x, dt, A, B, C, D=None, z=None, h0=None, *, dy, dh_final=None, lengths=None,
                               dt_softplus=False, dt_bias=None, want_carry_grads=False, workspace=None, out=None):
    """Gradients of m3_selective_scan for dy [Bt, L, D] (dense) and dh_final
    [Bt, D, N].  Returns a dict with dx, ddt, dA, dB, dC, dD, dz, ddt_bias
    (None where the input is) and, with want_carry_grads, dh0.  `out`:
    optional dict of preallocated tensors."""
    Bt, L, width = x.shape
    G, N = B.shape[-2:]
    dev, t = x.get_device(), x.dtype
    got = out or {}
    a = _lib.ScanBackwardArgs()
    a.fwd.Bt, a.fwd.L = Bt, L
    _scan_inputs(a.fwd, dev, (Bt, L), x, dt, A, B, C, D, z, dt_softplus, dt_bias)
    a.fwd.h0 = _dense(h0, _F32, (Bt, width, N), "h0", dev)
    a.fwd.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    a.dy = _dense(dy, t, (Bt, L, width), "dy", dev)
    a.dh_final = _dense(dh_final, _F32, (Bt, width, N), "dh_final", dev)
    out = {}
    rows, state = (Bt, L, width), (Bt, width, N)
    for k, like, shape, ty, wanted in (
            ("dx", x, rows, t, True), ("ddt", dt, rows, t, True), ("dA", A, (width, N), _F32, True), ("dB", B, B.shape, t, True),
            ("dC", C, B.shape, t, True), ("dD", D, (width,), _F32, D is not None), ("dz", z, rows, t, z is not None),
            ("ddt_bias", dt_bias, (width,), _F32, dt_bias is not None),
            ("dh0", x if h0 is None else h0, state, _F32, want_carry_grads or "dh0" in got)):
        out[k], at = _out(got.get(k), ty, shape, k, like, dev) if wanted else (None, None)
        setattr(a, k, at)
    workspace = _take_workspace("m3_selective_scan_backward", a, workspace, dev)
    _run_layer("m3_selective_scan_backward", a, dev)
    return out


def _gated_inputs(a, dev, x, z, w, groups, eps, gate_first):
    shape = x.shape
    n, width = len(shape) - 1, shape[-1]
    if width > _MAX or not -_MAX <= groups <= _MAX:
        _too_large(width, abs(groups))
    a.M, a.D, a.G, a.in_dtype = x.numel() // width if width else 0, width, groups, _dtype_code(x)
    a.gate_first, a.eps = 1 if gate_first else 0, eps
    a.x, a.x_ld = _rows(x, x.dtype, shape, n, "x", dev)
    a.z, a.z_ld = _rows(z, x.dtype, shape, n, "z", dev)
    a.w = _dense(w, _F32, (width,), "w", dev)


@_scoped
def m3_gated_norm(x, z=None, w=None, *, groups=1, eps=1e-6, gate_first=True, y=None):
    """Group RMS norm of rows with a SiLU gate: with gate_first v = x silu(z),
    y = v rsqrt(mean_group(v^2) + eps) w, else y = x rsqrt(mean_group(x^2) +
    eps) w silu(z).  x, z [..., D] (bf16 or fp32; rows may be slices of wider
    ones), w [D] fp32 (None: ones), `groups` equal groups.  Returns y (dense;
    may be given as x or z themselves where those are dense)."""
    dev = x.get_device()
    a = _lib.GatedNormArgs()
    _gated_inputs(a, dev, x, z, w, groups, eps, gate_first)
    y, a.y = _out(y, x.dtype, x.shape, "y", x, dev)
    _run_layer("m3_gated_norm", a, dev)
    return y


@_scoped
def m3_gated_norm_backward(x, z=None, w=None, *, dy, groups=1, eps=1e-6, gate_first=True, workspace=None, out=None):
    """Gradients of m3_gated_norm for dy (dense): a dict with dx, dz (None
    without gate) and dw (None without gain)."""
    dev, t = x.get_device(), x.dtype
    got = out or {}
    a = _lib.GatedNormBackwardArgs()
    _gated_inputs(a.fwd, dev, x, z, w, groups, eps, gate_first)
    a.dy = _dense(dy, t, x.shape, "dy", dev)
    out = dict(dx=None, dz=None, dw=None)
    out["dx"], a.dx = _out(got.get("dx"), t, x.shape, "dx", x, dev)
    if z is not None:
        out["dz"], a.dz = _out(got.get("dz"), t, x.shape, "dz", x, dev)
    if w is not None:
        out["dw"], a.dw = _out(got.get("dw"), _F32, x.shape[-1:], "dw", w, dev)
    workspace = _take_workspace("m3_gated_norm_backward", a, workspace, dev)
    _run_layer("m3_gated_norm_backward", a, dev)
    return out


@_scoped
def m3_residual_norm(x, residual=None, w=None, scale=None, *, eps=1e-6, y=None, residual_out=None, want_residual=True):
    """Residual sum and RMS norm: h = residual + scale x, y = h rsqrt(mean(h^2)
    + eps) w over rows of D.  x [..., D] (bf16 or fp32; rows may be slices of
    wider ones), residual of x's shape in x's type or fp32 (None: zeros), w and
    scale [D] fp32 (None: ones).  Returns a dict with y (x's type) and residual:
    h in the residual's type (residual_out may be `residual` itself)."""
    dev, t, shape = x.get_device(), x.dtype, x.shape
    width = shape[-1]
    like = residual if residual is not None else residual_out if residual_out is not None else x
    rt = like.dtype
    a = _lib.ResidualNormArgs()
    if width > _MAX:
        _too_large(width)
    a.M, a.D, a.in_dtype = x.numel() // width if width else 0, width, _dtype_code(x)
    a.res_dtype, a.eps = _lib.M3_F32 if rt == _F32 else a.in_dtype if rt == t else _dtype_code(like), eps
    a.x, a.x_ld = _rows(x, t, shape, len(shape) - 1, "x", dev)
    a.residual = _dense(residual, rt, shape, "residual", dev)
    a.scale = _dense(scale, _F32, (width,), "scale", dev)
    a.w = _dense(w, _F32, (width,), "w", dev)
    y, a.y = _out(y, t, shape, "y", x, dev)
    if want_residual or residual_out is not None:
        residual_out, a.residual_out = _out(residual_out, rt, shape, "residual_out", residual if residual is not None else x, dev)
    _run_layer("m3_residual_norm", a, dev)
    return dict(y=y, residual=residual_out)


@_scoped
def m3_residual_norm_backward(h, x=None, w=None, scale=None, *, dy, dresidual=None, eps=1e-6, workspace=None, out=None):
    """Gradients of m3_residual_norm at the stored sum h (its `residual`
    output) for dy and dresidual (the gradient that reaches h along the
    residual stream, h's type; None: zeros).  x is needed with scale only.
    Returns a dict with dresidual (h's type), dx (dy's type; the same tensor
    where scale is None and the types agree), dw and dscale (None where the
    parameter is).  out["dresidual"] may be `dresidual` itself."""
    dev, t, width = h.get_device(), dy.dtype, h.shape[-1]
    got = out or {}
    a = _lib.ResidualNormBackwardArgs()
    if width > _MAX:
        _too_large(width)
    a.M, a.D, a.in_dtype = h.numel() // width if width else 0, width, _dtype_code(dy)
    a.res_dtype, a.eps = _dtype_code(h), eps
    a.h = _dense(h, h.dtype, h.shape, "h", dev)
    a.x, a.x_ld = _rows(x, t, h.shape, h.dim() - 1, "x", dev)
    a.scale = _dense(scale, _F32, (width,), "scale", dev)
    a.w = _dense(w, _F32, (width,), "w", dev)
    a.dy = _dense(dy, t, h.shape, "dy", dev)
    a.dresidual_out = _dense(dresidual, h.dtype, h.shape, "dresidual", dev)
    out = dict(dresidual=None, dx=None, dw=None, dscale=None)
    out["dresidual"], a.dresidual = _out(got.get("dresidual"), h.dtype, h.shape, "dresidual", h, dev)
    if scale is not None or t != h.dtype or got.get("dx") is not None:
        out["dx"], a.dx = _out(got.get("dx"), t, h.shape, "dx", dy, dev)
    else:
        out["dx"] = out["dresidual"]
    if w is not None:
        out["dw"], a.dw = _out(got.get("dw"), _F32, (width,), "dw", w, dev)
    if scale is not None:
        out["dscale"], a.dscale = _out(got.get("dscale"), _F32, (width,), "dscale", scale, dev)
    workspace = _take_workspace("m3_residual_norm_backward", a, workspace, dev)
    _run_layer("m3_residual_norm_backward", a, dev)
    return out


# ---------------------------------------------------------------- linear attention
def _attention_inputs(a, dev, lead, q, k, v, log_decay, scale):
    """The inputs that linear attention, its backward and its step share."""
    t, n = q.dtype, len(lead)
    H, K = q.shape[n:]
    Hk, V = v.shape[n:]
    if max(H, Hk, K, V, *lead) > _MAX:
        _too_large(H, Hk, K, V, *lead)
    a.H, a.Hk, a.K, a.V, a.in_dtype = H, Hk, K, V, _dtype_code(q)
    a.scale = (K ** -0.5 if K else 0.0) if scale is None else scale
    a.q, a.q_ld = _rows(q, t, (*lead, H, K), n, "q", dev)
    a.k, a.k_ld = _rows(k, t, (*lead, Hk, K), n, "k", dev)
    a.v, a.v_ld = _rows(v, t, (*lead, Hk, V), n, "v", dev)
    a.log_decay = _dense(log_decay, _F32, (H,), "log_decay", dev)
    return H, Hk, K, V


@_scoped
def m3_linear_attention(q, k, v, log_decay, h0=None, *, scale=None, lengths=None, y=None, h_final=None, want_state=True,
                        workspace=None):
    """Linear attention with a constant decay for each head:
    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,  y_t = scale q_t^T S_t.
    q [Bt, L, H, K], k [Bt, L, Hk, K], v [Bt, L, Hk, V] (bf16 or fp32; tokens may be
    slices of wider rows; H / Hk heads of q share one of k and v), K and V in
    1..256; log_decay [H], h0 [Bt, H, K, V] fp32; scale: K^-1/2 if None; lengths
    [Bt] int32.  workspace: a uint8 device tensor, None to allocate one when the
    library asks for it, or False to run without (token axis not cut).  Returns a
    dict with y [Bt, L, H, V] (rows behind an item's length are left as they
    were) and h: the last state [Bt, H, K, V] (h_final may be `h0` itself)."""
    Bt, L = q.shape[:2]
    dev, t = q.get_device(), q.dtype
    a = _lib.LinearAttentionArgs()
    a.Bt, a.L = min(Bt, _MAX), min(L, _MAX)
    H, _, K, V = _attention_inputs(a, dev, (Bt, L), q, k, v, log_decay, scale)
    a.h0 = _dense(h0, _F32, (Bt, H, K, V), "h0", dev)
    a.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    y, a.y = _out(y, t, (Bt, L, H, V), "y", q, dev)
    if want_state or h_final is not None:
        h_final, a.h_final = _out(h_final, _F32, (Bt, H, K, V), "h_final", q if h0 is None else h0, dev)
    if workspace is not False:
        workspace = _take_workspace("m3_linear_attention", a, workspace, dev)
    _run_layer("m3_linear_attention", a, dev)
    return dict(y=y, h=h_final)


@_scoped
def m3_linear_attention_step(h, q, k, v, log_decay, *, scale=None, y=None, h_out=None):
    """One token of m3_linear_attention: q [Bt, H, K], k [Bt, Hk, K], v [Bt, Hk, V],
    h [Bt, H, K, V] fp32 updated in place (or read only, the new state going to
    h_out).  Returns y [Bt, H, V]."""
    Bt = q.shape[0]
    dev = h.get_device()
    a = _lib.LinearAttentionStepArgs()
    a.Bt = min(Bt, _MAX)
    H, _, K, V = _attention_inputs(a, dev, (Bt,), q, k, v, log_decay, scale)
    a.h = _dense(h, _F32, (Bt, H, K, V), "h", dev)
    a.h_out = _dense(h_out, _F32, (Bt, H, K, V), "h_out", dev)
    y, a.y = _out(y, q.dtype, (Bt, H, V), "y", q, dev)
    _run_layer("m3_linear_attention_step", a, dev)
    return y


@_scoped
def m3_linear_attention_backward(q, k, v, log_decay, h0=None, *, dy, dh_final=None, scale=None, lengths=None,
                                 want_carry_grads=False, workspace=None, out=None):
    """Gradients of m3_linear_attention for dy [Bt, L, H, V] (dense) and dh_final
    [Bt, H, K, V].  Returns a dict with dq, dk, dv (zero behind an item's length)
    and, with want_carry_grads, dh0.  log_decay is a constant.  `out`: optional
    dict of preallocated tensors."""
    Bt, L = q.shape[:2]
    dev, t = q.get_device(), q.dtype
    got = out or {}
    a = _lib.LinearAttentionBackwardArgs()
    a.fwd.Bt, a.fwd.L = min(Bt, _MAX), min(L, _MAX)
    H, Hk, K, V = _attention_inputs(a.fwd, dev, (Bt, L), q, k, v, log_decay, scale)
    state = (Bt, H, K, V)
    a.fwd.h0 = _dense(h0, _F32, state, "h0", dev)
    a.fwd.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)
    a.dy = _dense(dy, t, (Bt, L, H, V), "dy", dev)
    a.dh_final = _dense(dh_final, _F32, state, "dh_final", dev)
    out = dict(dq=None, dk=None, dv=None, dh0=None)
    out["dq"], a.dq = _out(got.get("dq"), t, (Bt, L, H, K), "dq", q, dev)
    out["dk"], a.dk = _out(got.get("dk"), t, (Bt, L, Hk, K), "dk", k, dev)
    out["dv"], a.dv = _out(got.get("dv"), t, (Bt, L, Hk, V), "dv", v, dev)
    if want_carry_grads or "dh0" in got:
        out["dh0"], a.dh0 = _out(got.get("dh0"), _F32, state, "dh0", q if h0 is None else h0, dev)
    workspace = _take_workspace("m3_linear_attention_backward", a, workspace, dev)
    _run_layer("m3_linear_attention_backward", a, dev)
    return out


def _rope_inputs(a, dev, q, k, q_w, k_w, freqs, positions, start, lengths, eps, norm, adjacent):
    """The inputs that the norm and rotation and its backward share."""
    Bt, L, H, D = q.shape
    t, Hk = q.dtype, 0 if k is None else k.shape[2]
    R = 0 if freqs is None else 2 * freqs.shape[0]
    if max(Bt, L, H, Hk, D, R) > _MAX:
        _too_large(Bt, L, H, Hk, D, R)
    if not -_MAX <= start <= _MAX:
        _too_large(abs(start))
    if k is None and k_w is not None:
        raise ValueError("k_w without k")
    a.Bt, a.L, a.H, a.Hk, a.D, a.R, a.in_dtype = Bt, L, H, Hk, D, R, _dtype_code(q)
    a.norm, a.adjacent, a.start, a.eps = 1 if norm else 0, 1 if adjacent else 0, start, eps
    a.q, a.q_ld = _rows(q, t, (Bt, L, H, D), 2, "q", dev)
    a.k, a.k_ld = _rows(k, t, (Bt, L, Hk, D), 2, "k", dev)
    a.q_w = _dense(q_w, _F32, (D,), "q_w", dev)
    a.k_w = _dense(k_w, _F32, (D,), "k_w", dev)
    a.freqs = _dense(freqs, _F32, (R // 2,), "freqs", dev)
    a.positions = _dense(positions, torch.int32, (Bt, L), "positions", dev)
    a.lengths = _dense(lengths, torch.int32, (Bt,), "lengths", dev)


@_scoped
def m3_qk_norm_rope(q, k=None, q_w=None, k_w=None, *, freqs=None, positions=None, start=0, lengths=None, eps=1e-6, norm=True,
                    adjacent=False, q_out=None, k_out=None):
    """RMS norm of queries and keys for each head and their rotation by position, in
    one pass: n = x rsqrt(mean(x^2) + eps) w (norm=False: n = x), then the first
    R = 2 len(freqs) elements in pairs (i, i + R/2), with `adjacent` (2i, 2i + 1):
    y0 = n0 cos a - n1 sin a, y1 = n1 cos a + n0 sin a, a = position freqs[i].  q
    [Bt, L, H, D], k [Bt, L, Hk, D] or None (bf16 or fp32; tokens may be slices of
    wider rows), D in 1..1024; q_w, k_w [D], freqs [R/2] fp32 (None: no rotation);
    positions [Bt, L] int32 (None: start + t); lengths [Bt] int32.  Returns a dict
    with q and k (dense; rows behind an item's length are left as they were; q_out
    and k_out may be q and k themselves where those are dense)."""
    dev, t = q.get_device(), q.dtype
    a = _lib.QkNormRopeArgs()
    _rope_inputs(a, dev, q, k, q_w, k_w, freqs, positions, start, lengths, eps, norm, adjacent)
    q_out, a.q_out = _out(q_out, t, q.shape, "q_out", q, dev)
    if k is not None:
        k_out, a.k_out = _out(k_out, t, k.shape, "k_out", k, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _run_layer("m3_qk_norm_rope", a, dev)
    return dict(q=q_out, k=k_out)


@_scoped
def m3_qk_norm_rope_backward(q, k=None, q_w=None, k_w=None, *, dq_out, dk_out=None, freqs=None, positions=None, start=0,
                             lengths=None, eps=1e-6, norm=True, adjacent=False, workspace=None, out=None):
    """Gradients of m3_qk_norm_rope for dq_out and dk_out (dense; the gradients of
    its outputs).  Returns a dict with dq, dk (None without k; zero behind an
    item's length), dq_w and dk_w (None where the gain is).  `out`: optional dict
    of preallocated tensors; its dq and dk may be dq_out and dk_out themselves."""
    dev, t = q.get_device(), q.dtype
    got = out or {}
    a = _lib.QkNormRopeBackwardArgs()
    _rope_inputs(a.fwd, dev, q, k, q_w, k_w, freqs, positions, start, lengths, eps, norm, adjacent)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out goes with k")
    a.dq_out = _dense(dq_out, t, q.shape, "dq_out", dev)
    a.dk_out = None if k is None else _dense(dk_out, t, k.shape, "dk_out", dev)
    out = dict(dq=None, dk=None, dq_w=None, dk_w=None)
    out["dq"], a.dq = _out(got.get("dq"), t, q.shape, "dq", q, dev)
    if k is not None:
        out["dk"], a.dk = _out(got.get("dk"), t, k.shape, "dk", k, dev)
    if q_w is not None:
        out["dq_w"], a.dq_w = _out(got.get("dq_w"), _F32, q_w.shape, "dq_w", q_w, dev)
    if k_w is not None:
        out["dk_w"], a.dk_w = _out(got.get("dk_w"), _F32, k_w.shape, "dk_w", k_w, dev)
    workspace = _take_workspace("m3_qk_norm_rope_backward", a, workspace, dev)
    _run_layer("m3_qk_norm_rope_backward", a, dev)
    return out
