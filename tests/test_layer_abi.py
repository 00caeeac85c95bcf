"""C-ABI contract of what stands around the scan in a layer (packed scan, short
convolution, residual rms norm), checked on the CPU: struct layout against the header,
workspace queries and every refused argument (all of them return before any HIP call;
the pointers are made up and never dereferenced)."""
import ctypes
import os
import subprocess

import pytest

import selective_state_space_83_amd as ssm
from selective_state_space_83_amd import layer as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GB = 1 << 30
BASE = 0x100000000
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIAS, WORKSPACE = range(7)
BIG = 1 << 62

STRUCTS = (("ssm_packed_scan_args_t", M.PackedScanArgs), ("ssm_packed_step_args_t", M.PackedStepArgs),
           ("ssm_packed_scan_bwd_args_t", M.PackedScanBwdArgs), ("ssm_short_conv_args_t", M.ShortConvArgs),
           ("ssm_short_conv_step_args_t", M.ShortConvStepArgs), ("ssm_short_conv_bwd_args_t", M.ShortConvBwdArgs),
           ("ssm_add_norm_args_t", M.AddNormArgs), ("ssm_add_norm_bwd_args_t", M.AddNormBwdArgs))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssm.LIB_PATH):
        from selective_state_space_83_amd import _build
        _build.build()
    return ssm.load_library()


def test_struct_layout_matches_header(tmp_path):
    lines = ['printf("%s sizeof %%zu\\n", sizeof(%s));' % (T, T) for T, _ in STRUCTS]
    lines += ['printf("%s %s %%zu\\n", offsetof(%s, %s));' % (T, f[0], T, f[0]) for T, cls in STRUCTS for f in cls._fields_]
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


def fill(a, **values):
    """Made-up pointers a GiB apart in every pointer field, then the values."""
    at = BASE
    for name, kind in a._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, at)
            at += GB
    for k, v in values.items():
        setattr(a, k, v)
    return a


ROWS = dict(x_stride=96, delta_stride=96, b_stride=16, c_stride=16)


def scan():
    return fill(M.PackedScanArgs(), tokens=3000, seqs=4, slots=6, dim=96, dstate=16, z_stride=96, workspace_bytes=GB, **ROWS)


def step():
    return fill(M.PackedStepArgs(), batch=4, slots=6, dim=96, dstate=16, z_stride=96, **ROWS)


def bwd():
    return fill(M.PackedScanBwdArgs(), tokens=300, seqs=4, dim=96, dstate=16, dy_stride=96, workspace_bytes=GB, **ROWS)


def conv():
    return fill(M.ShortConvArgs(), tokens=300, seqs=4, slots=6, channels=96, x_stride=96, taps=4, act=1)


def cstep():
    return fill(M.ShortConvStepArgs(), batch=4, slots=6, channels=96, x_stride=96, taps=4, act=1)


def cbwd():
    return fill(M.ShortConvBwdArgs(), tokens=300, seqs=4, channels=96, x_stride=96, dy_stride=96, taps=4, act=1, workspace_bytes=GB)


def norm():
    return fill(M.AddNormArgs(), rows=30, channels=96, x_stride=96, residual_stride=96, y_dtype=M.SSM_E4M3, block=32, eps=1e-5)


def nbwd():
    a = fill(M.AddNormBwdArgs(), rows=30, channels=96, sum_stride=96, dy_stride=96, dsum_stride=96, eps=1e-5, workspace_bytes=GB)
    a.dresidual = None
    return a


CALLS = {"scan": (scan, "ssm_packed_scan_fwd"), "step": (step, "ssm_packed_step"), "bwd": (bwd, "ssm_packed_scan_bwd"),
         "conv": (conv, "ssm_short_conv_fwd"), "cstep": (cstep, "ssm_short_conv_step"), "cbwd": (cbwd, "ssm_short_conv_bwd"),
         "norm": (norm, "ssm_add_norm_fwd"), "nbwd": (nbwd, "ssm_add_norm_bwd")}

REFUSED = [
    ("scan", SHAPE, dict(tokens=-1)), ("scan", SHAPE, dict(seqs=-1)), ("scan", SHAPE, dict(slots=-1)), ("scan", SHAPE, dict(dim=-1)),
    ("scan", SHAPE, dict(tokens=1 << 31)), ("scan", SHAPE, dict(seqs=1 << 31)), ("scan", SHAPE, dict(slots=1 << 31)),
    ("scan", SHAPE, dict(dim=BIG)), ("scan", UNSUPPORTED, dict(dstate=3)), ("scan", UNSUPPORTED, dict(dstate=0)),
    ("scan", UNSUPPORTED, dict(dstate=32)), ("scan", DTYPE, dict(dtype=2)), ("scan", DTYPE, dict(dtype=-1)), ("scan", DTYPE, dict(disc=2)),
    ("scan", UNSUPPORTED, dict(delta_softplus=2)), ("scan", UNSUPPORTED, dict(chunk_len=6)), ("scan", UNSUPPORTED, dict(chunk_len=-4)),
    ("scan", SHAPE, dict(x_stride=-1)), ("scan", SHAPE, dict(delta_stride=BIG)), ("scan", SHAPE, dict(z_stride=1 << 27)),
    ("scan", SHAPE, dict(b_stride=-1)), ("scan", SHAPE, dict(c_stride=BIG)), ("scan", SHAPE, dict(slot=None)),
    ("scan", UNSUPPORTED, dict(h0=None, h_last=None)), ("scan", NULL, dict(A=None)), ("scan", NULL, dict(offsets=None)),
    ("scan", NULL, dict(x=None)), ("scan", NULL, dict(delta=None)), ("scan", NULL, dict(Bm=None)), ("scan", NULL, dict(Cm=None)),
    ("scan", NULL, dict(y=None)), ("scan", UNSUPPORTED, dict(x=BASE + 2)), ("scan", UNSUPPORTED, dict(offsets=BASE + 2)),
    ("scan", UNSUPPORTED, dict(slot=BASE + 1)), ("scan", UNSUPPORTED, dict(h0=BASE + 2)), ("scan", UNSUPPORTED, dict(workspace=BASE + 64)),
    ("scan", WORKSPACE, dict(workspace=None)), ("scan", WORKSPACE, dict(workspace_bytes=16)), ("scan", ALIAS, dict(y="x")),
    ("scan", ALIAS, dict(y="Bm")), ("scan", ALIAS, dict(y="offsets")), ("scan", ALIAS, dict(h_last="A")), ("scan", ALIAS, dict(h_saved="h0")),
    ("scan", ALIAS, dict(h_last="y")), ("scan", ALIAS, dict(workspace="z")), ("scan", ALIAS, dict(h_saved="y")),
    ("step", SHAPE, dict(batch=-1)), ("step", SHAPE, dict(slots=-1)), ("step", SHAPE, dict(slot=None)), ("step", UNSUPPORTED, dict(reserved=1)),
    ("step", UNSUPPORTED, dict(dstate=5)), ("step", DTYPE, dict(dtype=3)), ("step", DTYPE, dict(disc=-1)), ("step", SHAPE, dict(x_stride=-2)),
    ("step", UNSUPPORTED, dict(delta_softplus=-1)), ("step", NULL, dict(h=None)), ("step", NULL, dict(y=None)), ("step", NULL, dict(Cm=None)),
    ("step", UNSUPPORTED, dict(h=BASE + 8)), ("step", UNSUPPORTED, dict(slot=BASE + 2)), ("step", ALIAS, dict(y="x")), ("step", ALIAS, dict(h="A")),
    ("step", ALIAS, dict(y="h")),
    ("bwd", SHAPE, dict(tokens=-1)), ("bwd", SHAPE, dict(seqs=-2)), ("bwd", UNSUPPORTED, dict(super_chunk=8)), ("bwd", UNSUPPORTED, dict(super_chunk=-16)),
    ("bwd", UNSUPPORTED, dict(reserved=1)), ("bwd", DTYPE, dict(dtype=7)), ("bwd", SHAPE, dict(dy_stride=-1)), ("bwd", SHAPE, dict(x_stride=1 << 25)),
    ("bwd", NULL, dict(h_saved=None)), ("bwd", NULL, dict(dA=None)), ("bwd", NULL, dict(dy=None)), ("bwd", NULL, dict(dB=None)), ("bwd", NULL, dict(offsets=None)),
    ("bwd", UNSUPPORTED, dict(dx=BASE + 1)), ("bwd", WORKSPACE, dict(workspace=None)), ("bwd", WORKSPACE, dict(workspace_bytes=0)),
    ("bwd", ALIAS, dict(dx="dy")), ("bwd", ALIAS, dict(dh0="dh_last")), ("bwd", ALIAS, dict(dB="dC")), ("bwd", ALIAS, dict(ddelta="workspace")),
    ("conv", SHAPE, dict(tokens=-1)), ("conv", SHAPE, dict(tokens=1 << 31)), ("conv", SHAPE, dict(channels=-1)), ("conv", SHAPE, dict(x_stride=-1)),
    ("conv", SHAPE, dict(x_stride=BIG)), ("conv", UNSUPPORTED, dict(taps=0)), ("conv", UNSUPPORTED, dict(taps=5)), ("conv", DTYPE, dict(act=2)),
    ("conv", DTYPE, dict(dtype=2)), ("conv", UNSUPPORTED, dict(reserved=1)), ("conv", SHAPE, dict(offsets=None, seqlen=7)),
    ("conv", SHAPE, dict(offsets=None, seqlen=-75)), ("conv", UNSUPPORTED, dict(state=None)), ("conv", SHAPE, dict(slot=None)),
    ("conv", NULL, dict(x=None)), ("conv", NULL, dict(weight=None)), ("conv", NULL, dict(y=None)), ("conv", UNSUPPORTED, dict(offsets=BASE + 1)),
    ("conv", UNSUPPORTED, dict(state=BASE + 2)), ("conv", ALIAS, dict(y="x")), ("conv", ALIAS, dict(state="x")), ("conv", ALIAS, dict(state="y")),
    ("conv", ALIAS, dict(y="resume")),
    ("cstep", SHAPE, dict(batch=-1)), ("cstep", SHAPE, dict(slot=None)), ("cstep", NULL, dict(state=None)), ("cstep", NULL, dict(y=None)),
    ("cstep", UNSUPPORTED, dict(taps=6)), ("cstep", ALIAS, dict(y="x")), ("cstep", ALIAS, dict(state="weight")), ("cstep", ALIAS, dict(y="state")),
    ("cbwd", SHAPE, dict(dy_stride=-1)), ("cbwd", SHAPE, dict(offsets=None, seqlen=0)), ("cbwd", NULL, dict(dx=None)), ("cbwd", NULL, dict(dy=None)),
    ("cbwd", WORKSPACE, dict(workspace=None)), ("cbwd", WORKSPACE, dict(workspace_bytes=8)), ("cbwd", UNSUPPORTED, dict(workspace=BASE + 4)),
    ("cbwd", UNSUPPORTED, dict(dweight=BASE + 2)), ("cbwd", ALIAS, dict(dx="dy")), ("cbwd", ALIAS, dict(dweight="dbias")), ("cbwd", ALIAS, dict(dx="x")),
    ("norm", SHAPE, dict(rows=-1)), ("norm", SHAPE, dict(rows=1 << 31)), ("norm", SHAPE, dict(channels=1 << 31)), ("norm", SHAPE, dict(x_stride=-1)),
    ("norm", SHAPE, dict(residual_stride=BIG)), ("norm", DTYPE, dict(dtype=2)), ("norm", DTYPE, dict(residual_dtype=1)), ("norm", DTYPE, dict(y_dtype=1)),
    ("norm", DTYPE, dict(y_dtype=3)), ("norm", UNSUPPORTED, dict(eps=-1.0)), ("norm", UNSUPPORTED, dict(eps=float("inf"))),
    ("norm", UNSUPPORTED, dict(eps=float("nan"))), ("norm", UNSUPPORTED, dict(block=48)), ("norm", UNSUPPORTED, dict(block=512)),
    ("norm", UNSUPPORTED, dict(block=-32)), ("norm", UNSUPPORTED, dict(y_dtype=0)), ("norm", UNSUPPORTED, dict(y_dtype=0, scale=None)),
    ("norm", UNSUPPORTED, dict(y_dtype=0, block=0)), ("norm", NULL, dict(x=None)), ("norm", NULL, dict(y=None)), ("norm", NULL, dict(scale=None)),
    ("norm", UNSUPPORTED, dict(x=BASE + 2)), ("norm", UNSUPPORTED, dict(scale=BASE + 2)), ("norm", ALIAS, dict(y="x")), ("norm", ALIAS, dict(y="residual")),
    ("norm", ALIAS, dict(sum="x")), ("norm", ALIAS, dict(sum="residual", residual_stride=128)), ("norm", ALIAS, dict(sum="y")),
    ("norm", ALIAS, dict(scale="weight")), ("norm", ALIAS, dict(scale="y")),
    ("nbwd", SHAPE, dict(dsum_stride=-1)), ("nbwd", DTYPE, dict(sum_dtype=1)), ("nbwd", UNSUPPORTED, dict(reserved=1)),
    ("nbwd", UNSUPPORTED, dict(dresidual=BASE + 40 * GB)), ("nbwd", UNSUPPORTED, dict(eps=float("nan"))), ("nbwd", NULL, dict(sum=None)),
    ("nbwd", NULL, dict(dy=None)), ("nbwd", NULL, dict(dx=None)), ("nbwd", WORKSPACE, dict(workspace=None)), ("nbwd", WORKSPACE, dict(workspace_bytes=4)),
    ("nbwd", UNSUPPORTED, dict(dweight=BASE + 2)), ("nbwd", ALIAS, dict(dx="dy")), ("nbwd", ALIAS, dict(dx="sum")), ("nbwd", ALIAS, dict(dweight="weight")),
    ("nbwd", ALIAS, dict(dweight="dx")),
]


@pytest.mark.parametrize("kind,status,fields", REFUSED, ids=lambda v: str(v))
def test_refused(lib, kind, status, fields):
    make, name = CALLS[kind]
    a = make()
    for k, v in fields.items():
        setattr(a, k, getattr(a, v) if isinstance(v, str) else v)
    assert getattr(lib, name)(ctypes.byref(a), None) == status, lib.ssm_last_error_message()
    assert lib.ssm_last_error_message()


@pytest.mark.parametrize("kind", list(CALLS))
def test_null_args(lib, kind):
    assert getattr(lib, CALLS[kind][1])(None, None) == NULL


def test_empty_problems_need_no_pointer(lib):
    """Nothing to do: no launch, whatever the pointers."""
    for a, name in ((M.PackedScanArgs(dstate=4), "ssm_packed_scan_fwd"), (M.PackedScanArgs(dstate=4, tokens=9, seqs=0, dim=8), "ssm_packed_scan_fwd"),
                    (M.PackedStepArgs(dstate=4), "ssm_packed_step"), (M.PackedScanBwdArgs(dstate=4, tokens=9), "ssm_packed_scan_bwd"),
                    (M.ShortConvArgs(taps=4), "ssm_short_conv_fwd"), (M.ShortConvStepArgs(taps=1, channels=8), "ssm_short_conv_step"),
                    (M.ShortConvBwdArgs(taps=4), "ssm_short_conv_bwd"), (M.AddNormArgs(rows=5), "ssm_add_norm_fwd"),
                    (M.AddNormBwdArgs(rows=5), "ssm_add_norm_bwd")):
        assert getattr(lib, name)(ctypes.byref(a), None) == OK, name


def test_workspace_queries(lib):
    size = lambda n, a: getattr(lib, n)(ctypes.byref(a))  # noqa: E731
    a = scan()
    assert size("ssm_packed_scan_workspace_size", a) > 0
    a.h_last = a.h0   # in place: the initial states that another workgroup would overwrite are kept
    more = size("ssm_packed_scan_workspace_size", a)
    a.h0 = None
    assert more > size("ssm_packed_scan_workspace_size", a)
    a.tokens = 32   # one chunk
    assert size("ssm_packed_scan_workspace_size", a) == 0
    # by the sizes alone: no address enters
    for n, make in (("ssm_packed_scan_bwd_workspace_size", bwd), ("ssm_short_conv_bwd_workspace_size", cbwd),
                    ("ssm_add_norm_bwd_workspace_size", nbwd)):
        a, b = make(), make()
        for f, kind in b._fields_:
            if kind is ctypes.c_void_p and getattr(b, f):
                setattr(b, f, getattr(b, f) + 4)
        assert size(n, a) == size(n, b) > 0
        assert getattr(lib, n)(None) == 0
    for n, make in (("ssm_short_conv_bwd_workspace_size", cbwd), ("ssm_add_norm_bwd_workspace_size", nbwd)):
        a = make()
        a.dweight = None
        if n.startswith("ssm_short"):
            a.dbias = None
        assert size(n, a) == 0
    for n, make, bad in (("ssm_packed_scan_workspace_size", scan, dict(tokens=-1)), ("ssm_packed_scan_bwd_workspace_size", bwd, dict(dstate=3)),
                         ("ssm_short_conv_bwd_workspace_size", cbwd, dict(taps=9)), ("ssm_add_norm_bwd_workspace_size", nbwd, dict(rows=BIG, channels=BIG))):
        a = make()
        for k, v in bad.items():
            setattr(a, k, v)
        assert size(n, a) == 0
        assert lib.ssm_last_error_message() == b""


def test_the_sum_may_take_the_residuals_place(lib):
    """An alias the checks let through: refused for another reason behind them."""
    a = norm()
    a.sum, a.y = a.residual, a.x
    assert lib.ssm_add_norm_fwd(ctypes.byref(a), None) == ALIAS
    assert b"residual" not in lib.ssm_last_error_message()
