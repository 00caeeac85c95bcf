"""What stands around the scan in a layer, for sequences of unequal lengths laid
one behind the other (contract: ``include/ssm_scan.h``).

    y, h_last = packed_scan(x, delta, A, B, C, offsets, D=None, h0=None, ...)
    y = packed_step(h, x, delta, A, B, C, D=None, slots=None, ...)      # h updated in place
    grads = packed_scan_bwd(x, delta, A, B, C, offsets, dy, h_saved, D=None, h0=None, ...)
    y = short_conv(x, weight, bias=None, offsets=None, act="silu", state=None, ...)
    y = short_conv_step(state, x, weight, bias=None, act="silu", slots=None)  # state updated in place
    grads = short_conv_bwd(x, weight, dy, bias=None, offsets=None, act="silu")
    y, total = add_rms_norm(x, residual, weight)
    q, scale, total = add_rms_norm_8bit(x, residual, weight, block=0)
    grads = add_rms_norm_bwd(total, dy, weight, dsum=None)

Packed tensors are (tokens, channels); sequence s holds the tokens offsets[s] to
offsets[s + 1] - 1 (int32, on the GPU).  Tokens of no sequence are not read and
their rows of y are left as they were (``y=`` gives the buffer).  States and windows
lie in a cache (slots, ...); ``slots`` (int32) names each sequence's entry, any
value outside the cache (-1) none: the sequence then starts from zero and keeps
nothing.  ``resume`` (bool) says which sequences take up their entry rather than start
from zero.  Inputs may be strided rows with contiguous channels (slices of a
projection's output).

Like the scan's binding, this module checks placement and shapes and marshals
pointers; the computation runs in the library's kernels on the current (or
given) stream.
"""
from __future__ import annotations

import ctypes

from . import SAVE_STRIDE, SSM_DISC_DELTA_B, SSM_DISC_ZOH, _on_stream, _raise_for, _torch, load_library
from .mixer import _code, _current, _dense, _norm_rows, _refuse, _rows, _workspace

SSM_E4M3 = 2
SSM_ACT_NONE = 0
SSM_ACT_SILU = 1

_i64, _i32, _ptr_t, _size = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


def _fields(kind, names):
    return [(n, kind) for n in names.split()]


class PackedScanArgs(ctypes.Structure):
    """Mirror of ssm_packed_scan_args_t."""
    _fields_ = (_fields(_i64, "tokens seqs slots dim dstate x_stride delta_stride z_stride b_stride c_stride")
                + _fields(_i32, "dtype disc delta_softplus chunk_len")
                + _fields(_ptr_t, "x delta A Bm Cm Dskip delta_bias z offsets slot resume h0 h_last h_saved y workspace")
                + [("workspace_bytes", _size)])


class PackedStepArgs(ctypes.Structure):
    """Mirror of ssm_packed_step_args_t."""
    _fields_ = (_fields(_i64, "batch slots dim dstate x_stride delta_stride z_stride b_stride c_stride")
                + _fields(_i32, "dtype disc delta_softplus reserved")
                + _fields(_ptr_t, "x delta A Bm Cm Dskip delta_bias z slot h y"))


class PackedScanBwdArgs(ctypes.Structure):
    """Mirror of ssm_packed_scan_bwd_args_t."""
    _fields_ = (_fields(_i64, "tokens seqs dim dstate x_stride delta_stride b_stride c_stride dy_stride")
                + _fields(_i32, "dtype disc super_chunk reserved")
                + _fields(_ptr_t, "x delta A Bm Cm Dskip offsets h0 h_saved dy dh_last dx ddelta dA dB dC dD dh0 workspace")
                + [("workspace_bytes", _size)])


class ShortConvArgs(ctypes.Structure):
    """Mirror of ssm_short_conv_args_t."""
    _fields_ = (_fields(_i64, "tokens seqs seqlen slots channels x_stride") + _fields(_i32, "dtype taps act reserved")
                + _fields(_ptr_t, "x weight bias offsets slot resume state y"))


class ShortConvStepArgs(ctypes.Structure):
    """Mirror of ssm_short_conv_step_args_t."""
    _fields_ = (_fields(_i64, "batch slots channels x_stride") + _fields(_i32, "dtype taps act reserved")
                + _fields(_ptr_t, "x weight bias slot state y"))


class ShortConvBwdArgs(ctypes.Structure):
    """Mirror of ssm_short_conv_bwd_args_t."""
    _fields_ = (_fields(_i64, "tokens seqs seqlen channels x_stride dy_stride") + _fields(_i32, "dtype taps act reserved")
                + _fields(_ptr_t, "x weight bias offsets dy dx dweight dbias workspace") + [("workspace_bytes", _size)])


class AddNormArgs(ctypes.Structure):
    """Mirror of ssm_add_norm_args_t."""
    _fields_ = (_fields(_i64, "rows channels block x_stride residual_stride") + _fields(_i32, "dtype residual_dtype y_dtype")
                + [("eps", ctypes.c_float)] + _fields(_ptr_t, "x residual weight sum y scale"))


class AddNormBwdArgs(ctypes.Structure):
    """Mirror of ssm_add_norm_bwd_args_t."""
    _fields_ = (_fields(_i64, "rows channels sum_stride dy_stride dsum_stride") + _fields(_i32, "dtype sum_dtype reserved")
                + [("eps", ctypes.c_float)] + _fields(_ptr_t, "sum dy dsum weight dx dresidual dweight workspace")
                + [("workspace_bytes", _size)])


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    P = ctypes.POINTER
    for name, args in (("ssm_packed_scan_fwd", PackedScanArgs), ("ssm_packed_step", PackedStepArgs),
                       ("ssm_packed_scan_bwd", PackedScanBwdArgs), ("ssm_short_conv_fwd", ShortConvArgs),
                       ("ssm_short_conv_step", ShortConvStepArgs), ("ssm_short_conv_bwd", ShortConvBwdArgs),
                       ("ssm_add_norm_fwd", AddNormArgs), ("ssm_add_norm_bwd", AddNormBwdArgs)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [P(args), ctypes.c_void_p]
    for name, args in (("ssm_packed_scan_workspace_size", PackedScanArgs),
                       ("ssm_packed_scan_bwd_workspace_size", PackedScanBwdArgs),
                       ("ssm_short_conv_bwd_workspace_size", ShortConvBwdArgs),
                       ("ssm_add_norm_bwd_workspace_size", AddNormBwdArgs)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_size_t, [P(args)]


# ---------------------------------------------------------------------------
# checks
# ---------------------------------------------------------------------------

def _rows2(t, name, shape, dtype, dev):
    """Address and row stride of a (rows, channels) input with contiguous channels."""
    ptr, s = _rows(t, name, shape, dtype, dev)
    return ptr, s[0] if shape[0] > 1 else shape[1]


def _even_rows(t, name, like, dev):
    """``_norm_rows``; a tensor without elements may have any strides."""
    if t.numel() == 0 and t.shape == like.shape and t.dtype is like.dtype and t.get_device() == dev:
        return t.data_ptr(), t.shape[-1]
    return _norm_rows(t, name, like, dev)


def _act(act):
    if act is None:
        return SSM_ACT_NONE
    if act == "silu":
        return SSM_ACT_SILU
    raise ValueError("act must be None or 'silu'")


def _offsets(a, offsets, dev):
    """Fills the offsets; returns the number of sequences."""
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be (sequences + 1,)")
    a.seqs = offsets.shape[0] - 1
    a.offsets = _dense(offsets, "offsets", offsets.shape, _torch().int32, dev)
    return a.seqs


def _places(a, slots, resume, seqs, dev):
    """Fills the slots and the resume flags of `seqs` sequences."""
    torch = _torch()
    a.slot = _dense(slots, "slots", (seqs,), torch.int32, dev)
    if resume is not None:
        dt = resume.dtype
        if dt is not torch.bool and dt is not torch.uint8:
            raise ValueError("resume must have dtype torch.bool")
        a.resume = _dense(resume, "resume", (seqs,), dt, dev)


def _recurrence(a, x, delta, A, B, C, D, zoh, dev):
    """Fills what the three calls of the recurrence share; returns (rows, dim), N and
    x's dtype."""
    if x.dim() != 2 or A.dim() != 2:
        raise ValueError("x must be (tokens, dim) and A (dim, N)")
    shape, dt, f32 = x.shape, x.dtype, _torch().float32
    dim, N = shape[1], A.shape[1]
    a.dim, a.dstate = dim, N
    a.dtype = _code(x, "x")
    a.disc = SSM_DISC_ZOH if zoh else SSM_DISC_DELTA_B
    a.x, a.x_stride = _rows2(x, "x", shape, dt, dev)
    a.delta, a.delta_stride = _rows2(delta, "delta", shape, dt, dev)
    narrow = (shape[0], N)
    a.Bm, a.b_stride = _rows2(B, "B", narrow, dt, dev)
    a.Cm, a.c_stride = _rows2(C, "C", narrow, dt, dev)
    a.A = _dense(A, "A", (dim, N), f32, dev)
    a.Dskip = _dense(D, "D", (dim,), f32, dev)
    return shape, N, dt


def _step_size(a, delta_bias, delta_softplus, z, shape, dt, dev):
    a.delta_bias = _dense(delta_bias, "delta_bias", shape[1:], _torch().float32, dev)
    a.delta_softplus = 1 if delta_softplus else 0
    if z is not None:
        a.z, a.z_stride = _rows2(z, "z", shape, dt, dev)


def packed_states_shape(tokens: int, dim: int, dstate: int) -> tuple:
    """Shape of the states a packed scan keeps for its backward pass (h_saved): the
    state before tokens 16, 32, ... below the number of tokens."""
    return (max(0, (tokens + SAVE_STRIDE - 1) // SAVE_STRIDE - 1), dim, dstate)


# ---------------------------------------------------------------------------
# packed scan
# ---------------------------------------------------------------------------

def packed_scan(x, delta, A, B, C, offsets, D=None, h0=None, h_last=None, slots=None, resume=None, zoh=False,
                delta_bias=None, delta_softplus=False, z=None, want_h_last=False, y=None, h_saved=None, chunk_len=0,
                workspace=None, stream=None):
    """The scan over packed sequences: x, delta, z (tokens, dim), B, C (tokens, N), A
    (dim, N).  Sequence s starts from entry slots[s] (s without slots) of h0 (float32,
    (slots, dim, N)), or from zero, and leaves its last state in that entry of h_last;
    ``h_last=h0`` updates a cache in place.  With ``want_h_last`` and no h_last one is
    made, a state per sequence.  ``h_saved`` (float32, ``packed_states_shape(...)``) is
    filled for ``packed_scan_bwd``.  Returns (y, h_last)."""
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = PackedScanArgs()
        shape, N, dt = _recurrence(a, x, delta, A, B, C, D, zoh, dev)
        a.tokens = shape[0]
        seqs = _offsets(a, offsets, dev)
        if h_last is None and want_h_last:
            if slots is not None and h0 is None:
                raise ValueError("with slots, h_last must be given")
            h_last = x.new_empty((seqs, shape[1], N) if h0 is None else h0.shape, dtype=torch.float32)
            if slots is not None:
                h_last.copy_(h0)   # the entries of no sequence
        cache = h0 if h0 is not None else h_last
        if cache is not None:
            if cache.dim() != 3:
                raise ValueError("states must be (slots, dim, N)")
            states = (cache.shape[0], shape[1], N)
            a.slots = states[0]
            a.h0 = _dense(h0, "h0", states, torch.float32, dev)
            a.h_last = _dense(h_last, "h_last", states, torch.float32, dev)
        _places(a, slots, resume, seqs, dev)
        _step_size(a, delta_bias, delta_softplus, z, shape, dt, dev)
        a.h_saved = _dense(h_saved, "h_saved", packed_states_shape(shape[0], shape[1], N), torch.float32, dev)
        if y is None:
            y = x.new_empty(shape)
        a.y = _dense(y, "y", shape, dt, dev)
        a.chunk_len = int(chunk_len)
        need = lib.ssm_packed_scan_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, x, dev)
        status = lib.ssm_packed_scan_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y, h_last


def packed_step(h, x, delta, A, B, C, D=None, slots=None, zoh=False, delta_bias=None, delta_softplus=False, z=None,
                y=None, stream=None):
    """One token for each row of a batch: x, delta, z (batch, dim), B, C (batch, N); row
    b's state is entry slots[b] (b without slots) of h (float32, (slots, dim, N)), updated
    in place.  Returns y (batch, dim)."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = PackedStepArgs()
        shape, N, dt = _recurrence(a, x, delta, A, B, C, D, zoh, dev)
        a.batch = shape[0]
        if h.dim() != 3:
            raise ValueError("h must be (slots, dim, N)")
        a.slots = h.shape[0]
        a.h = _dense(h, "h", (h.shape[0], shape[1], N), _torch().float32, dev)
        a.slot = _dense(slots, "slots", shape[:1], _torch().int32, dev)
        _step_size(a, delta_bias, delta_softplus, z, shape, dt, dev)
        if y is None:
            y = x.new_empty(shape)
        a.y = _dense(y, "y", shape, dt, dev)
        status = lib.ssm_packed_step(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def packed_scan_bwd(x, delta, A, B, C, offsets, dy, h_saved, D=None, h0=None, dh_last=None, zoh=False, want_dD=True,
                    want_dh0=True, super_chunk=0, workspace=None, stream=None) -> dict:
    """The gradients of sum(dy * y) + sum(dh_last * h_last) of ``packed_scan`` (a state
    per sequence, no softplus, bias or gate) from the states its call kept (h_saved): a
    dict of float32 tensors dx, ddelta, dA, dB, dC and, when asked, dD and dh0."""
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    f32 = torch.float32
    with _on_stream(stream):
        a = PackedScanBwdArgs()
        shape, N, dt = _recurrence(a, x, delta, A, B, C, D, zoh, dev)
        a.tokens = shape[0]
        seqs = _offsets(a, offsets, dev)
        states = (seqs, shape[1], N)
        a.dy, a.dy_stride = _rows2(dy, "dy", shape, dt, dev)
        a.h0 = _dense(h0, "h0", states, f32, dev)
        a.dh_last = _dense(dh_last, "dh_last", states, f32, dev)
        a.h_saved = _dense(h_saved, "h_saved", packed_states_shape(shape[0], shape[1], N), f32, dev)
        g = {"dx": x.new_empty(shape, dtype=f32), "ddelta": x.new_empty(shape, dtype=f32),
             "dA": A.new_empty(A.shape), "dB": x.new_empty((shape[0], N), dtype=f32),
             "dC": x.new_empty((shape[0], N), dtype=f32)}
        if want_dD:
            g["dD"] = x.new_empty(shape[1:], dtype=f32)
        if want_dh0:
            g["dh0"] = x.new_empty(states, dtype=f32)
        for name, t in g.items():
            setattr(a, name, t.data_ptr())
        a.super_chunk = int(super_chunk)
        need = lib.ssm_packed_scan_bwd_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, x, dev)
        status = lib.ssm_packed_scan_bwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return g


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------

def _conv_args(a, x, weight, bias, act, dev):
    if weight.dim() != 2:
        raise ValueError("weight must be (channels, K)")
    if x.dim() < 2:
        raise ValueError("x must be (tokens, channels) or (batch, L, channels)")
    f32, C = _torch().float32, x.shape[-1]
    a.channels, a.taps = C, weight.shape[1]
    a.dtype, a.act = _code(x, "x"), _act(act)
    a.x, a.x_stride = _even_rows(x, "x", x, dev)
    a.weight = _dense(weight, "weight", (C, weight.shape[1]), f32, dev)
    a.bias = _dense(bias, "bias", (C,), f32, dev)


def _conv_seqs(a, x, offsets, dev):
    if offsets is not None:
        if x.dim() != 2:
            raise ValueError("with offsets x must be (tokens, channels)")
        a.tokens = x.shape[0]
        return _offsets(a, offsets, dev)
    if x.dim() != 3:
        raise ValueError("without offsets x must be (batch, L, channels)")
    a.seqs, a.seqlen = x.shape[:2]
    a.tokens = a.seqs * a.seqlen
    return a.seqs


def short_conv(x, weight, bias=None, offsets=None, act="silu", state=None, slots=None, resume=None, y=None,
               stream=None):
    """Causal depthwise convolution, then silu (``act=None`` leaves it out): x (tokens,
    channels) with offsets, or (batch, L, channels); weight (channels, K <= 4), bias
    (channels,), float32.  ``state`` (float32, (slots, channels, K - 1), oldest input
    first) holds the inputs before each sequence and is moved on in place; without it
    sequences start from zeros.  Returns y like x."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = ShortConvArgs()
        _conv_args(a, x, weight, bias, act, dev)
        seqs = _conv_seqs(a, x, offsets, dev)
        if state is not None:
            if state.dim() != 3:
                raise ValueError("state must be (slots, channels, K - 1)")
            a.slots = state.shape[0]
            a.state = _dense(state, "state", (state.shape[0], x.shape[-1], weight.shape[1] - 1), _torch().float32, dev)
        _places(a, slots, resume, seqs, dev)
        if y is None:
            y = x.new_empty(x.shape)
        a.y = _dense(y, "y", x.shape, x.dtype, dev)
        status = lib.ssm_short_conv_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def short_conv_step(state, x, weight, bias=None, act="silu", slots=None, y=None, stream=None):
    """One token for each row of x (batch, channels): row b's window is entry slots[b] (b
    without slots) of state, moved on in place.  Returns y (batch, channels)."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = ShortConvStepArgs()
        if x.dim() != 2 or state.dim() != 3:
            raise ValueError("x must be (batch, channels) and state (slots, channels, K - 1)")
        _conv_args(a, x, weight, bias, act, dev)
        a.batch, a.slots = x.shape[0], state.shape[0]
        a.state = _dense(state, "state", (state.shape[0], x.shape[1], weight.shape[1] - 1), _torch().float32, dev)
        a.slot = _dense(slots, "slots", x.shape[:1], _torch().int32, dev)
        if y is None:
            y = x.new_empty(x.shape)
        a.y = _dense(y, "y", x.shape, x.dtype, dev)
        status = lib.ssm_short_conv_step(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def short_conv_bwd(x, weight, dy, bias=None, offsets=None, act="silu", want_dweight=True, want_dbias=True,
                   workspace=None, stream=None) -> dict:
    """The gradients of sum(dy * y) of ``short_conv`` without a state: dx (x's dtype) and,
    when asked, dweight and dbias (float32; dbias also where bias is None)."""
    lib = load_library()
    dev, handle = _current(stream)
    f32 = _torch().float32
    with _on_stream(stream):
        a = ShortConvBwdArgs()
        _conv_args(a, x, weight, bias, act, dev)
        _conv_seqs(a, x, offsets, dev)
        a.dy, a.dy_stride = _even_rows(dy, "dy", x, dev)
        g = {"dx": x.new_empty(x.shape)}
        if want_dweight:
            g["dweight"] = weight.new_empty(weight.shape)
        if want_dbias:
            g["dbias"] = x.new_empty(x.shape[-1:], dtype=f32)
        for name, t in g.items():
            setattr(a, name, t.data_ptr())
        need = lib.ssm_short_conv_bwd_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, x, dev)
        status = lib.ssm_short_conv_bwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return g


# ---------------------------------------------------------------------------
# residual and norm
# ---------------------------------------------------------------------------

def _wide(t, name, dtype):
    """dtype code of the residual stream: that of x, or float32."""
    code = _code(t, name)
    if t.dtype is not dtype and t.dtype is not _torch().float32:
        raise ValueError("%s must have x's dtype or float32" % name)
    return code


def _stream_rows(t, name, shape, dev):
    """Address and row stride of a tensor of the residual stream, its dtype its own."""
    if t.shape != shape or t.get_device() != dev:
        _refuse(t, name, shape, t.dtype, dev)
    return _even_rows(t, name, t, dev)


def _add_norm(x, residual, weight, eps, block, quant, y, total, keep, stream):
    torch = _torch()
    lib = load_library()
    dev, handle = _current(stream)
    f32 = torch.float32
    with _on_stream(stream):
        a = AddNormArgs()
        if x.dim() < 1:
            raise ValueError("x must be (..., channels)")
        shape, C = x.shape, x.shape[-1]
        a.channels, a.rows = C, x.numel() // C if C else 0
        a.block, a.eps = int(block), float(eps)
        a.dtype = a.residual_dtype = _code(x, "x")
        a.x, a.x_stride = _even_rows(x, "x", x, dev)
        a.weight = _dense(weight, "weight", (C,), f32, dev)
        if residual is None:
            if total is not None:
                raise ValueError("total goes with residual")
            total = x
        else:
            a.residual_dtype = _wide(residual, "residual", x.dtype)
            a.residual, a.residual_stride = _stream_rows(residual, "residual", shape, dev)
            if total is None and keep:
                total = residual.new_empty(shape)
            a.sum = _dense(total, "total", shape, residual.dtype, dev)
        if y is None:
            y = x.new_empty(shape, dtype=torch.float8_e4m3fn if quant else x.dtype)
        a.y = _dense(y, "y", shape, torch.float8_e4m3fn if quant else x.dtype, dev)
        a.y_dtype = SSM_E4M3 if quant else a.dtype
        scale = None
        if quant:
            scale = x.new_empty(shape[:-1] + (-(-C // block) if block > 0 else 1,), dtype=f32)
            a.scale = scale.data_ptr()
        status = lib.ssm_add_norm_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return (y, scale, total) if quant else (y, total)


def add_rms_norm(x, residual=None, weight=None, eps=1e-5, y=None, total=None, want_total=True, stream=None):
    """s = x + residual and y = s / sqrt(mean(s^2) + eps) * weight over the last
    dimension.  x (..., channels); residual like x, in x's dtype or float32, or None;
    weight float32 (channels,) or None.  Returns (y, total): total is s in the residual's
    dtype (``total=residual`` updates the stream in place), x itself without residual, None
    without ``want_total``."""
    return _add_norm(x, residual, weight, eps, 0, False, y, total, want_total, stream)


def add_rms_norm_8bit(x, residual=None, weight=None, eps=1e-5, block=0, y=None, total=None, want_total=True,
                      stream=None):
    """``add_rms_norm`` with y in 8 bits: returns (q, scale, total), q float8_e4m3fn with
    y ~ q * scale; scale float32 (..., ceil(channels / block)), one for each ``block``
    channels (32, 64, 128 or 256; 0: one for the row)."""
    return _add_norm(x, residual, weight, eps, block, True, y, total, want_total, stream)


def add_rms_norm_bwd(total, dy, weight=None, dsum=None, eps=1e-5, want_dweight=True, workspace=None, stream=None) -> dict:
    """The gradients of sum(dy * y) + sum(dsum * total) of ``add_rms_norm``, from its
    total: dx in dy's dtype, which is the residual's gradient too; where total has another
    dtype (float32) also dresidual in that; and, when asked, dweight (float32)."""
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        a = AddNormBwdArgs()
        if dy.dim() < 1:
            raise ValueError("dy must be (..., channels)")
        shape, C = dy.shape, dy.shape[-1]
        a.channels, a.rows, a.eps = C, dy.numel() // C if C else 0, float(eps)
        a.dtype, a.sum_dtype = _code(dy, "dy"), _wide(total, "total", dy.dtype)
        a.sum, a.sum_stride = _stream_rows(total, "total", shape, dev)
        a.dy, a.dy_stride = _even_rows(dy, "dy", dy, dev)
        if dsum is not None:
            a.dsum, a.dsum_stride = _even_rows(dsum, "dsum", total, dev)
        a.weight = _dense(weight, "weight", (C,), _torch().float32, dev)
        g = {"dx": dy.new_empty(shape)}
        if total.dtype is not dy.dtype:
            g["dresidual"] = total.new_empty(shape)
        if want_dweight:
            g["dweight"] = dy.new_empty((C,), dtype=_torch().float32)
        for name, t in g.items():
            setattr(a, name, t.data_ptr())
        need = lib.ssm_add_norm_bwd_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, need, workspace, dy, dev)
        status = lib.ssm_add_norm_bwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return g
