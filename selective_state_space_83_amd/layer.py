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
    grads = add_rms_norm_bwd(x, dy, weight, dsum=None, residual=None)

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
    f = lib.ssm_add_norm_bwd_residual
    f.restype, f.argtypes = ctypes.c_int, [P(AddNormBwdArgs), ctypes.c_void_p, _i64, ctypes.c_void_p]
    for name, args in (("ssm_packed_scan_workspace_size", PackedScanArgs),
                       ("ssm_packed_scan_bwd_workspace_size", PackedScanBwdArgs),
                       ("ssm_short_conv_bwd_workspace_size", ShortConvBwdArgs),
                       ("ssm_add_norm_bwd_workspace_size", AddNormBwdArgs)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_size_t, [P(args)]


# ---------------------------------------------------------------------------
# checks (small calls take as long as the host's part: each argument structure is
# filled in one go, which takes a third of the time of its fields one by one)
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


def _out(out, name, like, shape, dtype, dev, torch):
    """An output and its address: the one given, checked, or a new one."""
    if out is None:
        # (dense, whatever like's strides; a third of the time of torch.empty)
        if dtype is like.dtype and shape == like.shape:
            out = torch.empty_like(like, memory_format=torch.contiguous_format)
        else:
            out = torch.empty(shape, dtype=dtype, device=like.device)
        return out, out.data_ptr()
    return out, _dense(out, name, shape, dtype, dev)


def _act(act):
    if act is None:
        return SSM_ACT_NONE
    if act == "silu":
        return SSM_ACT_SILU
    raise ValueError("act must be None or 'silu'")


def _offsets(offsets, int32, dev):
    """Address of the offsets, and the number of sequences."""
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError("offsets must be (sequences + 1,)")
    return _dense(offsets, "offsets", shape, int32, dev), shape[0] - 1


def _resume(resume, seqs, torch, dev):
    if resume is None:
        return None
    dt = resume.dtype
    if dt is not torch.bool and dt is not torch.uint8:
        raise ValueError("resume must have dtype torch.bool")
    return _dense(resume, "resume", (seqs,), dt, dev)


def _recurrence(x, delta, A, B, C, D, zoh, f32, dev):
    """What the three calls of the recurrence share: the shape of x, N, x's dtype, then
    (strides), (dtype and discretization codes), (addresses)."""
    shape, coef = x.shape, A.shape
    if len(shape) != 2 or len(coef) != 2:
        raise ValueError("x must be (tokens, dim) and A (dim, N)")
    dt, dim, N = x.dtype, shape[1], coef[1]
    code = _code(x, "x")
    narrow = (shape[0], N)
    px, xs = _rows2(x, "x", shape, dt, dev)
    pd, ds = _rows2(delta, "delta", shape, dt, dev)
    pb, bs = _rows2(B, "B", narrow, dt, dev)
    pc, cs = _rows2(C, "C", narrow, dt, dev)
    return (shape, N, dt, (xs, ds, bs, cs), (code, SSM_DISC_ZOH if zoh else SSM_DISC_DELTA_B),
            (px, pd, _dense(A, "A", (dim, N), f32, dev), pb, pc, _dense(D, "D", (dim,), f32, dev)))


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
    made, a state per sequence (with slots a copy of h0 to begin with).  ``h_saved``
    (float32, ``packed_states_shape(...)``) is filled for ``packed_scan_bwd``.  Returns
    (y, h_last)."""
    torch = _torch()
    f32, int32 = torch.float32, torch.int32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        shape, N, dt, (xs, ds, bs, cs), codes, (px, pd, pA, pB, pC, pD) = _recurrence(x, delta, A, B, C, D, zoh, f32, dev)
        tokens, dim = shape
        p_off, seqs = _offsets(offsets, int32, dev)
        if h_last is None and want_h_last:
            if slots is not None and h0 is None:
                raise ValueError("with slots, h_last must be given")
            h_last = torch.empty((seqs, dim, N) if h0 is None else h0.shape, dtype=f32, device=x.device)
            if slots is not None:
                h_last.copy_(h0)   # the entries of no sequence
        entries = 0
        p_h0 = p_last = None
        cache = h0 if h0 is not None else h_last
        if cache is not None:
            if cache.dim() != 3:
                raise ValueError("states must be (slots, dim, N)")
            entries = cache.shape[0]
            states = (entries, dim, N)
            p_h0 = _dense(h0, "h0", states, f32, dev)
            p_last = p_h0 if h_last is h0 else _dense(h_last, "h_last", states, f32, dev)
        p_z, zs = (None, 0) if z is None else _rows2(z, "z", shape, dt, dev)
        y, p_y = _out(y, "y", x, shape, dt, dev, torch)
        a = PackedScanArgs(
            tokens, seqs, entries, dim, N, xs, ds, zs, bs, cs, *codes, 1 if delta_softplus else 0, int(chunk_len),
            px, pd, pA, pB, pC, pD, _dense(delta_bias, "delta_bias", (dim,), f32, dev), p_z, p_off,
            _dense(slots, "slots", (seqs,), int32, dev), _resume(resume, seqs, torch, dev), p_h0, p_last,
            _dense(h_saved, "h_saved", packed_states_shape(tokens, dim, N), f32, dev), p_y)
        arg = ctypes.byref(a)
        workspace = _workspace(a, lib.ssm_packed_scan_workspace_size(arg), workspace, x, dev)
        status = lib.ssm_packed_scan_fwd(arg, handle)
    _raise_for(lib, status)
    return y, h_last


def packed_step(h, x, delta, A, B, C, D=None, slots=None, zoh=False, delta_bias=None, delta_softplus=False, z=None,
                y=None, stream=None):
    """One token for each row of a batch: x, delta, z (batch, dim), B, C (batch, N); row
    b's state is entry slots[b] (b without slots) of h (float32, (slots, dim, N)), updated
    in place.  Returns y (batch, dim)."""
    torch = _torch()
    f32 = torch.float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        shape, N, dt, (xs, ds, bs, cs), codes, (px, pd, pA, pB, pC, pD) = _recurrence(x, delta, A, B, C, D, zoh, f32, dev)
        batch, dim = shape
        if h.dim() != 3:
            raise ValueError("h must be (slots, dim, N)")
        entries = h.shape[0]
        p_z, zs = (None, 0) if z is None else _rows2(z, "z", shape, dt, dev)
        y, p_y = _out(y, "y", x, shape, dt, dev, torch)
        a = PackedStepArgs(
            batch, entries, dim, N, xs, ds, zs, bs, cs, *codes, 1 if delta_softplus else 0, 0,
            px, pd, pA, pB, pC, pD, _dense(delta_bias, "delta_bias", (dim,), f32, dev), p_z,
            _dense(slots, "slots", (batch,), torch.int32, dev), _dense(h, "h", (entries, dim, N), f32, dev), p_y)
        status = lib.ssm_packed_step(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def packed_scan_bwd(x, delta, A, B, C, offsets, dy, h_saved, D=None, h0=None, dh_last=None, zoh=False, want_dD=True,
                    want_dh0=True, super_chunk=0, workspace=None, stream=None) -> dict:
    """The gradients of sum(dy * y) + sum(dh_last * h_last) of ``packed_scan`` (a state
    per sequence, no softplus, bias or gate) from the states its call kept (h_saved): a
    dict of float32 tensors dx, ddelta, dA, dB, dC and, when asked, dD and dh0."""
    torch = _torch()
    f32 = torch.float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        shape, N, dt, (xs, ds, bs, cs), codes, (px, pd, pA, pB, pC, pD) = _recurrence(x, delta, A, B, C, D, zoh, f32, dev)
        tokens, dim = shape
        p_off, seqs = _offsets(offsets, torch.int32, dev)
        states = (seqs, dim, N)
        p_dy, ys = _rows2(dy, "dy", shape, dt, dev)
        g = {"dx": torch.empty(shape, dtype=f32, device=x.device), "ddelta": torch.empty(shape, dtype=f32, device=x.device),
             "dA": A.new_empty(A.shape), "dB": torch.empty((tokens, N), dtype=f32, device=x.device),
             "dC": torch.empty((tokens, N), dtype=f32, device=x.device)}
        if want_dD:
            g["dD"] = torch.empty((dim,), dtype=f32, device=x.device)
        if want_dh0:
            g["dh0"] = torch.empty(states, dtype=f32, device=x.device)
        a = PackedScanBwdArgs(
            tokens, seqs, dim, N, xs, ds, bs, cs, ys, *codes, int(super_chunk), 0,
            px, pd, pA, pB, pC, pD, p_off, _dense(h0, "h0", states, f32, dev),
            _dense(h_saved, "h_saved", packed_states_shape(tokens, dim, N), f32, dev), p_dy,
            _dense(dh_last, "dh_last", states, f32, dev), g["dx"].data_ptr(), g["ddelta"].data_ptr(), g["dA"].data_ptr(),
            g["dB"].data_ptr(), g["dC"].data_ptr(), g["dD"].data_ptr() if want_dD else None,
            g["dh0"].data_ptr() if want_dh0 else None)
        arg = ctypes.byref(a)
        workspace = _workspace(a, lib.ssm_packed_scan_bwd_workspace_size(arg), workspace, x, dev)
        status = lib.ssm_packed_scan_bwd(arg, handle)
    _raise_for(lib, status)
    return g


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------

def _conv_args(x, weight, bias, f32, dev):
    """channels, K, x's stride and dtype code, and the addresses of x, weight and bias."""
    taps, shape = weight.shape, x.shape
    if len(taps) != 2:
        raise ValueError("weight must be (channels, K)")
    if len(shape) < 2:
        raise ValueError("x must be (tokens, channels) or (batch, L, channels)")
    channels = shape[-1]
    code = _code(x, "x")
    px, xs = _even_rows(x, "x", x, dev)
    return (channels, taps[1], xs, code,
            (px, _dense(weight, "weight", (channels, taps[1]), f32, dev), _dense(bias, "bias", (channels,), f32, dev)))


def _conv_seqs(x, offsets, int32, dev):
    """tokens, sequences, tokens of each (0 with offsets) and the offsets' address."""
    shape = x.shape
    if offsets is not None:
        if len(shape) != 2:
            raise ValueError("with offsets x must be (tokens, channels)")
        p_off, seqs = _offsets(offsets, int32, dev)
        return shape[0], seqs, 0, p_off
    if len(shape) != 3:
        raise ValueError("without offsets x must be (batch, L, channels)")
    return shape[0] * shape[1], shape[0], shape[1], None


def short_conv(x, weight, bias=None, offsets=None, act="silu", state=None, slots=None, resume=None, y=None,
               stream=None):
    """Causal depthwise convolution, then silu (``act=None`` leaves it out): x (tokens,
    channels) with offsets, or (batch, L, channels); weight (channels, K <= 4), bias
    (channels,), float32.  ``state`` (float32, (slots, channels, K - 1), oldest input
    first) holds the inputs before each sequence and is moved on in place; without it
    sequences start from zeros.  Returns y like x."""
    torch = _torch()
    f32, int32 = torch.float32, torch.int32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        channels, K, xs, code, where = _conv_args(x, weight, bias, f32, dev)
        tokens, seqs, seqlen, p_off = _conv_seqs(x, offsets, int32, dev)
        entries, p_state = 0, None
        if state is not None:
            if state.dim() != 3:
                raise ValueError("state must be (slots, channels, K - 1)")
            entries = state.shape[0]
            p_state = _dense(state, "state", (entries, channels, K - 1), f32, dev)
        y, p_y = _out(y, "y", x, x.shape, x.dtype, dev, torch)
        a = ShortConvArgs(tokens, seqs, seqlen, entries, channels, xs, code, K, _act(act), 0, *where, p_off,
                          _dense(slots, "slots", (seqs,), int32, dev), _resume(resume, seqs, torch, dev), p_state, p_y)
        status = lib.ssm_short_conv_fwd(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def short_conv_step(state, x, weight, bias=None, act="silu", slots=None, y=None, stream=None):
    """One token for each row of x (batch, channels): row b's window is entry slots[b] (b
    without slots) of state, moved on in place.  Returns y (batch, channels)."""
    torch = _torch()
    f32 = torch.float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        if x.dim() != 2 or state.dim() != 3:
            raise ValueError("x must be (batch, channels) and state (slots, channels, K - 1)")
        channels, K, xs, code, where = _conv_args(x, weight, bias, f32, dev)
        batch, entries = x.shape[0], state.shape[0]
        y, p_y = _out(y, "y", x, x.shape, x.dtype, dev, torch)
        a = ShortConvStepArgs(batch, entries, channels, xs, code, K, _act(act), 0, *where,
                              _dense(slots, "slots", (batch,), torch.int32, dev),
                              _dense(state, "state", (entries, channels, K - 1), f32, dev), p_y)
        status = lib.ssm_short_conv_step(ctypes.byref(a), handle)
    _raise_for(lib, status)
    return y


def short_conv_bwd(x, weight, dy, bias=None, offsets=None, act="silu", want_dweight=True, want_dbias=True,
                   workspace=None, stream=None) -> dict:
    """The gradients of sum(dy * y) of ``short_conv`` without a state: dx (x's dtype) and,
    when asked, dweight and dbias (float32; dbias also where bias is None)."""
    torch = _torch()
    f32 = torch.float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        channels, K, xs, code, where = _conv_args(x, weight, bias, f32, dev)
        tokens, seqs, seqlen, p_off = _conv_seqs(x, offsets, torch.int32, dev)
        p_dy, ys = _even_rows(dy, "dy", x, dev)
        g = {"dx": x.new_empty(x.shape)}
        if want_dweight:
            g["dweight"] = weight.new_empty(weight.shape)
        if want_dbias:
            g["dbias"] = torch.empty((channels,), dtype=f32, device=x.device)
        a = ShortConvBwdArgs(tokens, seqs, seqlen, channels, xs, ys, code, K, _act(act), 0, *where, p_off, p_dy,
                             g["dx"].data_ptr(), g["dweight"].data_ptr() if want_dweight else None,
                             g["dbias"].data_ptr() if want_dbias else None)
        arg = ctypes.byref(a)
        workspace = _workspace(a, lib.ssm_short_conv_bwd_workspace_size(arg), workspace, x, dev)
        status = lib.ssm_short_conv_bwd(arg, handle)
    _raise_for(lib, status)
    return g


# ---------------------------------------------------------------------------
# residual and norm
# ---------------------------------------------------------------------------

def _wide(t, name, dtype, f32):
    """dtype code of the residual stream: that of x, or float32."""
    code = _code(t, name)
    if t.dtype is not dtype and t.dtype is not f32:
        raise ValueError("%s must have x's dtype or float32" % name)
    return code


def _stream_rows(t, name, shape, dev):
    """Address and row stride of a tensor of the residual stream, its dtype its own."""
    if t.shape != shape or t.get_device() != dev:
        _refuse(t, name, shape, t.dtype, dev)
    return _even_rows(t, name, t, dev)


def _add_norm(x, residual, weight, eps, block, quant, y, total, keep, stream):
    torch = _torch()
    f32 = torch.float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        shape, dt = x.shape, x.dtype
        if len(shape) < 1:
            raise ValueError("x must be (..., channels)")
        C = shape[-1]
        block = int(block)
        code = wide = _code(x, "x")
        px, xs = _even_rows(x, "x", x, dev)
        p_res, rs, p_sum = None, 0, None
        if residual is None:
            if total is not None:
                raise ValueError("total goes with residual")
            total = x
        else:
            wide = _wide(residual, "residual", dt, f32)
            p_res, rs = _stream_rows(residual, "residual", shape, dev)
            if total is not None or keep:
                total, p_sum = _out(total, "total", x, shape, residual.dtype, dev, torch)
        ydt = torch.float8_e4m3fn if quant else dt
        y, p_y = _out(y, "y", x, shape, ydt, dev, torch)
        scale, p_scale = None, None
        if quant:
            scale, p_scale = _out(None, "scale", x, shape[:-1] + (-(-C // block) if block > 0 else 1,), f32, dev, torch)
        a = AddNormArgs(x.numel() // C if C else 0, C, block, xs, rs, code, wide, SSM_E4M3 if quant else code, eps, px, p_res,
                        _dense(weight, "weight", (C,), f32, dev), p_sum, p_y, p_scale)
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


def add_rms_norm_bwd(total, dy, weight=None, dsum=None, eps=1e-5, want_dweight=True, workspace=None, stream=None,
                     residual=None) -> dict:
    """The gradients of sum(dy * y) + sum(dsum * total) of ``add_rms_norm``: with
    ``residual`` (which then has not been updated in place) from x, given as ``total``, and
    residual; else from its total.  y comes from the sum before it is rounded to total's
    dtype, so a bfloat16 total gives other gradients, those at the rounded sum (dweight off by
    about 2e-3 of its norm); a float32 total gives the same.  Returns dx in dy's dtype,
    which is the residual's gradient too; where the residual (or total) has another dtype
    (float32) also dresidual in that; and, when asked, dweight (float32)."""
    f32 = _torch().float32
    lib = load_library()
    dev, handle = _current(stream)
    with _on_stream(stream):
        shape, dt = dy.shape, dy.dtype
        if len(shape) < 1:
            raise ValueError("dy must be (..., channels)")
        C = shape[-1]
        code = _code(dy, "dy")
        if residual is None:
            kept, wide = total, _wide(total, "total", dt, f32)
            p_sum, ss = _stream_rows(total, "total", shape, dev)
        else:
            kept, wide = residual, _wide(residual, "residual", dt, f32)
            p_sum, ss = _even_rows(total, "x", dy, dev)
            p_res, rs = _stream_rows(residual, "residual", shape, dev)
        p_dy, ds = _even_rows(dy, "dy", dy, dev)
        p_dsum, gs = (None, 0) if dsum is None else _even_rows(dsum, "dsum", kept, dev)
        g = {"dx": dy.new_empty(shape)}
        both = kept.dtype is not dt
        if both:
            g["dresidual"] = kept.new_empty(shape)
        if want_dweight:
            g["dweight"] = dy.new_empty((C,), dtype=f32)
        a = AddNormBwdArgs(dy.numel() // C if C else 0, C, ss, ds, gs, code, wide, 0, eps, p_sum, p_dy, p_dsum,
                           _dense(weight, "weight", (C,), f32, dev), g["dx"].data_ptr(),
                           g["dresidual"].data_ptr() if both else None, g["dweight"].data_ptr() if want_dweight else None)
        arg = ctypes.byref(a)
        workspace = _workspace(a, lib.ssm_add_norm_bwd_workspace_size(arg), workspace, dy, dev)
        if residual is None:
            status = lib.ssm_add_norm_bwd(arg, handle)
        else:
            status = lib.ssm_add_norm_bwd_residual(arg, p_res, rs, handle)
    _raise_for(lib, status)
    return g
