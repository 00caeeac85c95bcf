"""A library built before the present sources: the binding says to rebuild it,
whether its version differs or it only lacks later entry points."""
import os
import subprocess

import pytest

import selective_state_space_83_amd as ssm

LATER = ("ssm_decay_attn_fwd", "ssm_group_norm_bwd")


def stub(tmp_path, names, version):
    src = tmp_path / "stub.c"
    src.write_text("int ssm_abi_version(void) { return %d; }\n" % version
                   + "".join("void %s(void) {}\n" % n for n in names if n != "ssm_abi_version"))
    out = tmp_path / "libstub.so"
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    return str(out)


@pytest.mark.parametrize("names,version", [
    ([n for n in ssm.EXPORTS if n not in LATER], ssm.ABI_VERSION),
    ([n for n in ssm.EXPORTS if n not in LATER], ssm.ABI_VERSION - 1),
    (ssm.EXPORTS, ssm.ABI_VERSION - 1),
])
def test_older_library_says_rebuild(tmp_path, names, version):
    with pytest.raises(RuntimeError, match="rebuild it"):
        ssm.load_library(stub(tmp_path, names, version))


def test_every_declared_entry_point_is_listed():
    if not os.path.exists(ssm.LIB_PATH):
        from selective_state_space_83_amd import _build
        _build.build()
    lib = ssm.load_library()
    assert all(hasattr(lib, n) for n in ssm.EXPORTS)
