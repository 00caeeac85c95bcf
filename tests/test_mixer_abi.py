"""C-ABI contract of the head-decay mixer (decay attention and the group norm),
checked on the CPU: struct layout against the header, workspace queries and
every refused argument (all of them return before any HIP call; the pointers
are made up and never dereferenced)."""
import ctypes
import os
import subprocess

import pytest

import selective_state_space_83_amd as ssm
from selective_state_space_83_amd import mixer as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GB = 1 << 30
BASE = 0x100000000

STRUCTS = (("ssm_decay_attn_args_t", M.DecayAttnArgs), ("ssm_decay_attn_step_args_t", M.DecayAttnStepArgs),
           ("ssm_decay_attn_bwd_args_t", M.DecayAttnBwdArgs), ("ssm_group_norm_args_t", M.GroupNormArgs),
           ("ssm_group_norm_bwd_args_t", M.GroupNormBwdArgs))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        from selective_state_space_83_amd import _build
        _build.build()
    return ssm.load_library()


def test_struct_layout_matches_header(tmp_path):
    lines = ['printf("%s sizeof %%zu\\n", sizeof(%s));' % (T, T) for T, _ in STRUCTS]
    lines += ['printf("%s %s %%zu\\n", offsetof(%s, %s));' % (T, f[0], T, f[0])
              for T, cls in STRUCTS for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"ssm_scan.h\"\nint main(void) {\n%s\n"
                   "return 0; }\n" % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for T, cls in STRUCTS:
        assert got[(T, "sizeof")] == ctypes.sizeof(cls), T
        for f in cls._fields_:
            assert got[(T, f[0])] == getattr(cls, f[0]).offset, (T, f[0])


def _pointers(a, names):
    for i, n in enumerate(names):
        setattr(a, n, BASE + i * GB)


def fwd(B=2, L=64, H=4, Hk=2, dk=32, dv=16, dtype=ssm.SSM_F32):
    a = M.DecayAttnArgs()
    a.batch, a.seqlen, a.heads, a.key_heads, a.key_dim, a.value_dim = B, L, H, Hk, dk, dv
    a.dtype = a.decay_dtype = dtype
    a.q_stride[:] = a.k_stride[:] = (L * Hk * dk, Hk * dk, dk)
    a.v_stride[:] = (L * H * dv, H * dv, dv)
    a.decay_stride[:] = (L * H, H, 1)
    _pointers(a, ["q", "k", "v", "log_decay", "lengths", "h0", "h_last", "o", "workspace"])
    a.workspace_bytes = GB
    return a


def step(B=2, H=4, Hk=2, dk=32, dv=16):
    a = M.DecayAttnStepArgs()
    a.batch, a.heads, a.key_heads, a.key_dim, a.value_dim = B, H, Hk, dk, dv
    a.q_stride[:] = a.k_stride[:] = (Hk * dk, dk)
    a.v_stride[:] = (H * dv, dv)
    a.decay_stride[:] = (H, 1)
    _pointers(a, ["q", "k", "v", "log_decay", "h", "o"])
    return a


def bwd(**kw):
    f = fwd(**kw)
    a = M.DecayAttnBwdArgs()
    for n in ("batch", "seqlen", "heads", "key_heads", "key_dim", "value_dim", "dtype", "decay_dtype"):
        setattr(a, n, getattr(f, n))
    for n in ("q_stride", "k_stride", "v_stride", "decay_stride"):
        getattr(a, n)[:] = getattr(f, n)[:]
    a.dout_stride[:] = f.v_stride[:]
    _pointers(a, ["q", "k", "v", "log_decay", "dout", "lengths", "h0", "dh_last", "dq", "dk", "dv", "dlog_decay",
                  "dh0", "workspace"])
    a.workspace_bytes = GB
    return a


def norm(rows=8, C=64, G=4, mode=M.SSM_NORM_GATE, cls=M.GroupNormArgs):
    a = cls()
    a.rows, a.channels, a.groups, a.x_stride, a.z_stride = rows, C, G, C, C
    a.mode, a.eps = mode, 1e-5
    names = ["x", "z", "weight", "bias"]
    if cls is M.GroupNormArgs:
        names += ["y"]
    else:
        a.dy_stride, a.workspace_bytes = C, GB
        names += ["dy", "dx", "dz", "dweight", "dbias", "workspace"]
    _pointers(a, names)
    if mode < M.SSM_NORM_GATE:
        a.z = None
        if cls is not M.GroupNormArgs:
            a.dz = None
    return a


def nbwd(**kw):
    return norm(cls=M.GroupNormBwdArgs, **kw)


CALLS = {"fwd": (fwd, "ssm_decay_attn_fwd"), "step": (step, "ssm_decay_attn_step"), "bwd": (bwd, "ssm_decay_attn_bwd"),
         "norm": (norm, "ssm_group_norm_fwd"), "nbwd": (nbwd, "ssm_group_norm_bwd")}


def refused(lib, kind, status, **fields):
    make, name = CALLS[kind]
    a = make()
    for f, v in fields.items():
        if isinstance(v, tuple):
            getattr(a, f)[:] = v
        else:
            setattr(a, f, v)
    got = getattr(lib, name)(ctypes.byref(a), None)
    assert got == status, (kind, fields, got, lib.ssm_last_error_message())
    assert lib.ssm_last_error_message()


def test_null_arguments(lib):
    for make, name in CALLS.values():
        assert getattr(lib, name)(None, None) == ssm.SSM_ERR_NULL
    for name in ("ssm_decay_attn_workspace_size", "ssm_decay_attn_bwd_workspace_size",
                 "ssm_group_norm_bwd_workspace_size"):
        assert getattr(lib, name)(None) == 0


@pytest.mark.parametrize("kind,names", [
    ("fwd", ["q", "k", "v", "log_decay", "o"]), ("step", ["q", "k", "v", "log_decay", "h", "o"]),
    ("bwd", ["q", "k", "v", "log_decay", "dout", "dq", "dk", "dv", "dlog_decay"]), ("norm", ["x", "z", "y"]),
    ("nbwd", ["x", "z", "dy", "dx", "dz"])])
def test_required_pointers(lib, kind, names):
    for n in names:
        refused(lib, kind, ssm.SSM_ERR_NULL, **{n: None})


@pytest.mark.parametrize("kind", ["fwd", "step", "bwd"])
def test_attention_sizes_and_types(lib, kind):
    for f in ("batch", "heads", "key_heads"):
        refused(lib, kind, ssm.SSM_ERR_SHAPE, **{f: -1})
    if kind != "step":
        refused(lib, kind, ssm.SSM_ERR_SHAPE, seqlen=-1)
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, span=-64)
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, span=65)
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, reserved=1)
        refused(lib, kind, ssm.SSM_ERR_SHAPE, seqlen=1 << 60)
    for f in ("key_dim", "value_dim"):
        refused(lib, kind, ssm.SSM_ERR_SHAPE, **{f: 0})
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, **{f: 257})
    refused(lib, kind, ssm.SSM_ERR_SHAPE, key_heads=3)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, key_heads=0)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, batch=1 << 62)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, batch=1 << 31)
    refused(lib, kind, ssm.SSM_ERR_DTYPE, dtype=2)
    refused(lib, kind, ssm.SSM_ERR_DTYPE, decay_dtype=-1)
    bad = (-1, 1, 1) if kind != "step" else (-1, 1)
    big = (1 << 62, 1, 1) if kind != "step" else (1 << 62, 1)
    for f in ["q_stride", "k_stride", "v_stride", "decay_stride"] + (["dout_stride"] if kind == "bwd" else []):
        refused(lib, kind, ssm.SSM_ERR_SHAPE, **{f: bad})
        refused(lib, kind, ssm.SSM_ERR_SHAPE, **{f: big})


@pytest.mark.parametrize("kind,names", [
    ("fwd", ["q", "k", "v", "log_decay", "o", "h0", "h_last", "lengths"]),
    ("step", ["q", "k", "v", "log_decay", "h", "o"]),
    ("bwd", ["q", "k", "v", "log_decay", "dout", "dq", "dk", "dv", "dlog_decay", "h0", "dh_last", "dh0", "workspace"]),
    ("norm", ["x", "z", "y", "weight", "bias"]),
    ("nbwd", ["x", "z", "dy", "dx", "dz", "weight", "bias", "dweight", "dbias", "workspace"])])
def test_alignment(lib, kind, names):
    for n in names:
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, **{n: BASE + 60 * GB + 2})


@pytest.mark.parametrize("kind,outs,ins", [
    ("fwd", ["o", "h_last"], ["q", "k", "v", "log_decay", "h0", "lengths"]),
    ("step", ["o", "h"], ["q", "k", "v", "log_decay"]),
    ("bwd", ["dq", "dk", "dv", "dlog_decay", "dh0", "workspace"],
     ["q", "k", "v", "log_decay", "dout", "h0", "dh_last", "lengths"]),
    ("norm", ["y"], ["x", "z", "weight", "bias"]),
    ("nbwd", ["dx", "dz", "dweight", "dbias", "workspace"], ["x", "z", "dy", "weight", "bias"])])
def test_overlaps(lib, kind, outs, ins):
    a = CALLS[kind][0]()
    for o in outs:
        for i in ins + [x for x in outs if x != o]:
            refused(lib, kind, ssm.SSM_ERR_ALIAS, **{o: getattr(a, i)})


def test_overlap_counts_strides(lib):
    """The last row of a strided input lies far behind its first."""
    a = fwd()
    refused(lib, "fwd", ssm.SSM_ERR_ALIAS, q_stride=(1 << 26, 64, 32), o=a.q + (1 << 28))
    refused(lib, "norm", ssm.SSM_ERR_ALIAS, x_stride=1 << 26, y=norm().x + 7 * (1 << 28))


def test_workspaces(lib):
    a = bwd()
    need = lib.ssm_decay_attn_bwd_workspace_size(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    refused(lib, "bwd", ssm.SSM_ERR_WORKSPACE, workspace_bytes=need - 1)
    refused(lib, "bwd", ssm.SSM_ERR_WORKSPACE, workspace=None)
    b = nbwd()
    need = lib.ssm_group_norm_bwd_workspace_size(ctypes.byref(b))
    assert need > 0
    refused(lib, "nbwd", ssm.SSM_ERR_WORKSPACE, workspace_bytes=need - 1)
    refused(lib, "nbwd", ssm.SSM_ERR_WORKSPACE, workspace=None)
    b.dweight = b.dbias = None
    assert lib.ssm_group_norm_bwd_workspace_size(ctypes.byref(b)) == 0
    for bad in (dict(key_dim=0), dict(heads=3), dict(batch=-1)):
        for make, name in ((fwd, "ssm_decay_attn_workspace_size"), (bwd, "ssm_decay_attn_bwd_workspace_size")):
            c = make()
            for f, v in bad.items():
                setattr(c, f, v)
            assert getattr(lib, name)(ctypes.byref(c)) == 0


@pytest.mark.parametrize("kind", ["norm", "nbwd"])
def test_norm_sizes_and_modes(lib, kind):
    refused(lib, kind, ssm.SSM_ERR_SHAPE, rows=-1)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, channels=-1)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, groups=0)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, groups=5)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, rows=1 << 60)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, x_stride=-1)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, x_stride=1 << 62)
    refused(lib, kind, ssm.SSM_ERR_SHAPE, z_stride=-1)
    refused(lib, kind, ssm.SSM_ERR_DTYPE, dtype=2)
    refused(lib, kind, ssm.SSM_ERR_DTYPE, mode=4)
    refused(lib, kind, ssm.SSM_ERR_DTYPE, mode=-1)
    refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, rms=2)
    refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, mode=M.SSM_NORM_SILU)   # with z
    for eps in (-1e-5, float("nan"), float("inf")):
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, eps=eps)
    if kind == "nbwd":
        refused(lib, kind, ssm.SSM_ERR_SHAPE, dy_stride=-1)
        refused(lib, kind, ssm.SSM_ERR_UNSUPPORTED, mode=M.SSM_NORM_PLAIN, z=None)   # with dz


def test_empty_calls_do_nothing(lib):
    a = fwd(B=0)
    assert lib.ssm_decay_attn_fwd(ctypes.byref(a), None) == ssm.SSM_OK
    a = fwd(L=0)
    a.h_last = None
    assert lib.ssm_decay_attn_fwd(ctypes.byref(a), None) == ssm.SSM_OK
    s = step(B=0)
    assert lib.ssm_decay_attn_step(ctypes.byref(s), None) == ssm.SSM_OK
    b = bwd(B=0)
    assert lib.ssm_decay_attn_bwd(ctypes.byref(b), None) == ssm.SSM_OK
    n = norm(rows=0)
    assert lib.ssm_group_norm_fwd(ctypes.byref(n), None) == ssm.SSM_OK
    n = nbwd(rows=0)
    n.dweight = n.dbias = None
    assert lib.ssm_group_norm_bwd(ctypes.byref(n), None) == ssm.SSM_OK
