"""Decay attention and the group norm that follows it: the part of the binding
for the head-decay mixer (contract: ``include/ssm_scan.h``).

    o, h_last = decay_attn(q, k, v, log_decay, h0=None, lengths=None)
    o = decay_attn_step(h, q, k, v, log_decay)          # h updated in place
    grads = decay_attn_bwd(q, k, v, log_decay, dout, h0=None, dh_last=None)
    y = group_norm(x, groups, weight, bias, z=None, act=None)
    grads = group_norm_bwd(x, dy, groups, weight, bias, z=None, act=None)

Decay attention is linear attention with a decay for each head: per batch row
and head  S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t.  Shapes:
q, k (batch, L, key_heads, key_dim); v, o (batch, L, heads, value_dim);
log_decay (batch, L, heads); states (batch, heads, key_dim, value_dim)
float32; lengths (batch,) int32 on the GPU.  Inputs may be strided views with a
contiguous last dimension (slices of one projection's output, broadcasts).

The group norm normalizes each token's channels in groups, scales and shifts
them, and applies silu (``act="silu"``) or the gate silu(z), after the norm or
before it (``gate_first``); ``rms`` leaves the mean in.

Like the scan's binding, this module checks placement and shapes and marshals
pointers; the computation runs in the library's kernels on the current (or
given) stream.
"""
from __future__ import annotations

import ctypes

from . import SSM_BF16, SSM_F32, _on_stream, _raise_for, _torch, load_library

SSM_NORM_PLAIN = 0
SSM_NORM_SILU = 1
SSM_NORM_GATE = 2
SSM_NORM_GATE_FIRST = 3

_i64, _i32, _ptr_t = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
_s2, _s3 = _i64 * 2, _i64 * 3


class DecayAttnArgs(ctypes.Structure):
    """Mirror of ssm_decay_attn_args_t."""
    _fields_ = [
        ("batch", _i64), ("seqlen", _i64), ("heads", _i64), ("key_heads", _i64),
        ("key_dim", _i64), ("value_dim", _i64),
        ("dtype", _i32), ("decay_dtype", _i32), ("span", _i32), ("reserved", _i32),
        ("q", _ptr_t), ("k", _ptr_t), ("v", _ptr_t), ("log_decay", _ptr_t),
        ("q_stride", _s3), ("k_stride", _s3), ("v_stride", _s3), ("decay_stride", _s3),
        ("lengths", _ptr_t), ("h0", _ptr_t), ("h_last", _ptr_t), ("o", _ptr_t),
        ("workspace", _ptr_t), ("workspace_bytes", ctypes.c_size_t),
    ]


class DecayAttnStepArgs(ctypes.Structure):
    """Mirror of ssm_decay_attn_step_args_t."""
    _fields_ = [
        ("batch", _i64), ("heads", _i64), ("key_heads", _i64), ("key_dim", _i64),
        ("value_dim", _i64), ("dtype", _i32), ("decay_dtype", _i32),
        ("q", _ptr_t), ("k", _ptr_t), ("v", _ptr_t), ("log_decay", _ptr_t),
        ("q_stride", _s2), ("k_stride", _s2), ("v_stride", _s2), ("decay_stride", _s2),
        ("h", _ptr_t), ("o", _ptr_t),
    ]


class DecayAttnBwdArgs(ctypes.Structure):
    """Mirror of ssm_decay_attn_bwd_args_t."""
    _fields_ = [
        ("batch", _i64), ("seqlen", _i64), ("heads", _i64), ("key_heads", _i64),
        ("key_dim", _i64), ("value_dim", _i64),
        ("dtype", _i32), ("decay_dtype", _i32), ("span", _i32), ("reserved", _i32),
        ("q", _ptr_t), ("k", _ptr_t), ("v", _ptr_t), ("log_decay", _ptr_t), ("dout", _ptr_t),
        ("q_stride", _s3), ("k_stride", _s3), ("v_stride", _s3), ("decay_stride", _s3),
        ("dout_stride", _s3),
        ("lengths", _ptr_t), ("h0", _ptr_t), ("dh_last", _ptr_t),
        ("dq", _ptr_t), ("dk", _ptr_t), ("dv", _ptr_t), ("dlog_decay", _ptr_t), ("dh0", _ptr_t),
        ("workspace", _ptr_t), ("workspace_bytes", ctypes.c_size_t),
    ]


class GroupNormArgs(ctypes.Structure):
    """Mirror of ssm_group_norm_args_t."""
    _fields_ = [
        ("rows", _i64), ("channels", _i64), ("groups", _i64), ("x_stride", _i64),
        ("z_stride", _i64), ("dtype", _i32), ("mode", _i32), ("rms", _i32),
        ("eps", ctypes.c_float), ("x", _ptr_t), ("z", _ptr_t), ("weight", _ptr_t),
        ("bias", _ptr_t), ("y", _ptr_t),
    ]


class GroupNormBwdArgs(ctypes.Structure):
    """Mirror of ssm_group_norm_bwd_args_t."""
    _fields_ = [
        ("rows", _i64), ("channels", _i64), ("groups", _i64), ("x_stride", _i64),
        ("z_stride", _i64), ("dy_stride", _i64), ("dtype", _i32), ("mode", _i32), ("rms", _i32),
        ("eps", ctypes.c_float), ("x", _ptr_t), ("z", _ptr_t), ("weight", _ptr_t),
        ("bias", _ptr_t), ("dy", _ptr_t), ("dx", _ptr_t), ("dz", _ptr_t), ("dweight", _ptr_t),
        ("dbias", _ptr_t), ("workspace", _ptr_t), ("workspace_bytes", ctypes.c_size_t),
    ]


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    P = ctypes.POINTER
    for name, args in (("ssm_decay_attn_fwd", DecayAttnArgs),
                       ("ssm_decay_attn_step", DecayAttnStepArgs),
                       ("ssm_decay_attn_bwd", DecayAttnBwdArgs),
                       ("ssm_group_norm_fwd", GroupNormArgs),
                       ("ssm_group_norm_bwd", GroupNormBwdArgs)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [P(args), ctypes.c_void_p]
    for name, args in (("ssm_decay_attn_workspace_size", DecayAttnArgs),
                       ("ssm_decay_attn_bwd_workspace_size", DecayAttnBwdArgs),
                       ("ssm_group_norm_bwd_workspace_size", GroupNormBwdArgs)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_size_t, [P(args)]


# ---------------------------------------------------------------------------
# checks (on the path of single-token calls, where the host's time is the
# call's: one test in the common case, the reason worked out only on failure)
# ---------------------------------------------------------------------------

def _code(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return SSM_BF16
    if t.dtype is torch.float32:
        return SSM_F32
    raise ValueError("unsupported dtype %s of %s (float32 or bfloat16)" % (t.dtype, name))


def _current(stream):
    """Index of the device the call runs on, the given stream's or the current one,
    and the handle of the stream to launch on."""
    torch = _torch()
    if stream is not None:
        return stream.device.index, stream.cuda_stream
    dev = torch.cuda.current_device()
    # the same handle without a Stream object around it, where this PyTorch has it
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return dev, raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _refuse(t, name, shape, dtype, dev):
    if t.shape != shape:
        raise ValueError("%s must be %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype is not dtype:
        raise ValueError("%s must have dtype %s" % (name, dtype))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    raise ValueError("%s is on cuda:%d but the current device is cuda:%d" % (name, t.get_device(), dev))


def _rows(t, name, shape, dtype, dev):
    """Address and outer strides of an input whose last dimension is contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, shape, dtype, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return t.data_ptr(), s[:-1]


def _dense(t, name, shape, dtype, dev):
    """Address of a contiguous tensor, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _workspace(args, need, workspace, like, dev):
    """Fills the workspace fields; returns the tensor to keep until the launch."""
    torch = _torch()
    if need == 0:
        return None
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    args.workspace = _dense(workspace, "workspace", workspace.shape, torch.uint8, dev)
    args.workspace_bytes = workspace.numel()
    return workspace


def _attn_inputs(a, q, k, v, log_decay, step, dev):
    """Fills sizes, dtypes, inputs and strides; returns the shapes of v and of the
    state."""
    vs, qs = v.shape, q.shape
    rank = 3 if step else 4
    if len(vs) != rank or len(qs) != rank:
        raise ValueError("q and v must have %d dimensions" % rank)
    dt, outer = q.dtype, vs[:-1]
    key_shape = vs[:-2] + qs[-2:]
    a.batch, a.heads, a.value_dim = vs[0], vs[-2], vs[-1]
    a.key_heads, a.key_dim = qs[-2], qs[-1]
    if not step:
        a.seqlen = vs[1]
    a.dtype, a.decay_dtype = _code(q, "q"), _code(log_decay, "log_decay")
    a.q, a.q_stride[:] = _rows(q, "q", key_shape, dt, dev)
    a.k, a.k_stride[:] = _rows(k, "k", key_shape, dt, dev)
    a.v, a.v_stride[:] = _rows(v, "v", vs, dt, dev)
    if log_decay.shape != outer or log_decay.get_device() != dev:
        _refuse(log_decay, "log_decay", outer, log_decay.dtype, dev)
    a.log_decay = log_decay.data_ptr()
    a.decay_stride[:] = log_decay.stride()
    return vs, (vs[0], vs[-2], qs[-1], vs[-1])


# ---------------------------------------------------------------------------
# decay attention
# ---------------------------------------------------------------------------

def decay_attn(q, k, v, log_decay, h0=None, lengths=None, want_h_last=True, o=None, h_last=None,
               span=0, workspace=None, stream=None):
    """Decay attention over whole sequences.  Returns (o, h_last); h_last is
    None when want_h_last is False and no h_last tensor is passed.  ``lengths``
    gives each row's number of tokens (o is 0 past it); ``span`` the tokens per
    span of the time axis (0: the library's plan)."""
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    f32 = torch.float32
    with _on_stream(stream):
        a = DecayAttnArgs()
        shape, state = _attn_inputs(a, q, k, v, log_decay, False, dev)
        if o is None:
            o = v.new_empty(shape)
        if h_last is None and want_h_last:
            h_last = v.new_empty(state, dtype=f32)
        a.o = _dense(o, "o", shape, v.dtype, dev)
        a.h0 = _dense(h0, "h0", state, f32, dev)
        a.h_last = _dense(h_last, "h_last", state, f32, dev)
        a.lengths = _dense(lengths, "lengths", shape[:1], torch.int32, dev)
        a.span = int(span)
        need = lib.ssm_decay_attn_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, v, dev)
        status = lib.ssm_decay_attn_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return o, h_last


def decay_attn_step(h, q, k, v, log_decay, o=None, stream=None):
    """One token per sequence: h (float32, (batch, heads, key_dim, value_dim))
    is updated in place; q, k (batch, key_heads, key_dim), v (batch, heads,
    value_dim), log_decay (batch, heads).  Returns o (batch, heads, value_dim)."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = DecayAttnStepArgs()
        shape, state = _attn_inputs(a, q, k, v, log_decay, True, dev)
        if o is None:
            o = v.new_empty(shape)
        a.h = _dense(h, "h", state, _torch().float32, dev)
        a.o = _dense(o, "o", shape, v.dtype, dev)
        status = lib.ssm_decay_attn_step(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return o


def decay_attn_bwd(q, k, v, log_decay, dout, h0=None, dh_last=None, lengths=None, want_dh0=True,
                   span=0, workspace=None, stream=None) -> dict:
    """The gradients of sum(dout * o) + sum(dh_last * h_last) of ``decay_attn``.
    Returns a dict of dense tensors: dq, dk, dv (the inputs' dtype), dlog_decay
    (its dtype) and, when asked, dh0 (float32).  A gradient has its input's full
    shape: sum it over the dimensions that a broadcast input repeats."""
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = DecayAttnBwdArgs()
        shape, state = _attn_inputs(a, q, k, v, log_decay, False, dev)
        a.dout, a.dout_stride[:] = _rows(dout, "dout", shape, v.dtype, dev)
        g = {"dq": q.new_empty(q.shape), "dk": q.new_empty(q.shape), "dv": v.new_empty(shape),
             "dlog_decay": log_decay.new_empty(log_decay.shape)}
        if want_dh0:
            g["dh0"] = v.new_empty(state, dtype=torch.float32)
        for name, t in g.items():
            setattr(a, name, t.data_ptr())
        a.h0 = _dense(h0, "h0", state, torch.float32, dev)
        a.dh_last = _dense(dh_last, "dh_last", state, torch.float32, dev)
        a.lengths = _dense(lengths, "lengths", shape[:1], torch.int32, dev)
        a.span = int(span)
        need = lib.ssm_decay_attn_bwd_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, v, dev)
        status = lib.ssm_decay_attn_bwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return g


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def _norm_rows(t, name, like, dev):
    """Address and row stride of a (..., channels) tensor whose rows are evenly
    spaced."""
    shape = like.shape
    if t.shape != shape or t.dtype is not like.dtype or t.get_device() != dev:
        _refuse(t, name, shape, like.dtype, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError("the channels of %s must be contiguous" % name)
    if len(shape) == 2:
        return t.data_ptr(), s[0] if shape[0] > 1 else shape[1]
    row, span = None, 0
    for n, st in zip(reversed(shape[:-1]), reversed(s[:-1])):
        if n == 1:
            continue
        if row is None:
            row = st
        elif st != span:
            raise ValueError("the rows of %s must be evenly spaced" % name)
        span = st * n
    return t.data_ptr(), shape[-1] if row is None else row


def _norm_args(a, x, groups, weight, bias, z, act, gate_first, rms, eps, dev):
    if x.dim() < 1:
        raise ValueError("x must be (..., channels)")
    if act not in (None, "silu"):
        raise ValueError("act must be None or 'silu'")
    if act is not None and z is not None:
        raise ValueError("act and z exclude each other")
    if gate_first and z is None:
        raise ValueError("gate_first needs z")
    C = x.shape[-1]
    a.channels, a.groups = C, int(groups)
    a.rows = x.numel() // C if C else 0
    a.dtype = _code(x, "x")
    a.mode = (SSM_NORM_SILU if act else SSM_NORM_PLAIN) if z is None else (
        SSM_NORM_GATE_FIRST if gate_first else SSM_NORM_GATE)
    a.rms, a.eps = (1 if rms else 0), float(eps)
    a.x, a.x_stride = _norm_rows(x, "x", x, dev)
    if z is not None:
        a.z, a.z_stride = _norm_rows(z, "z", x, dev)
    f32 = _torch().float32
    a.weight = _dense(weight, "weight", (C,), f32, dev)
    a.bias = _dense(bias, "bias", (C,), f32, dev)


def group_norm(x, groups, weight=None, bias=None, z=None, act=None, gate_first=False, rms=False,
               eps=1e-5, y=None, stream=None):
    """Group norm over the channels of each token of x (..., channels), then
    silu (``act="silu"``) or the gate silu(z); with ``gate_first`` x silu(z) is
    normalized instead.  weight and bias are float32 (channels,) or None."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = GroupNormArgs()
        _norm_args(a, x, groups, weight, bias, z, act, gate_first, rms, eps, dev)
        if y is None:
            y = x.new_empty(x.shape)
        a.y = _dense(y, "y", x.shape, x.dtype, dev)
        status = lib.ssm_group_norm_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def group_norm_bwd(x, dy, groups, weight=None, bias=None, z=None, act=None, gate_first=False,
                   rms=False, eps=1e-5, want_dweight=True, want_dbias=True, workspace=None,
                   stream=None) -> dict:
    """The gradients of sum(dy * y) of ``group_norm``: a dict of dense tensors
    dx, dz (with z; both of x's dtype) and, when asked, dweight and dbias
    (float32)."""
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = GroupNormBwdArgs()
        _norm_args(a, x, groups, weight, bias, z, act, gate_first, rms, eps, dev)
        a.dy, a.dy_stride = _norm_rows(dy, "dy", x, dev)
        g = {"dx": x.new_empty(x.shape)}
        if z is not None:
            g["dz"] = x.new_empty(x.shape)
        for name, want in (("dweight", want_dweight), ("dbias", want_dbias)):
            if want:
                g[name] = x.new_empty(x.shape[-1:], dtype=torch.float32)
        for name, t in g.items():
            setattr(a, name, t.data_ptr())
        need = lib.ssm_group_norm_bwd_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, x, dev)
        status = lib.ssm_group_norm_bwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return g
