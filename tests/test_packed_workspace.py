"""The packed scan's workspace goes by sizes and by which arguments are given, not by
their addresses: one sized for a cache that is copied serves a cache updated in place
(CPU; the pointers are made up and never dereferenced)."""
import ctypes

import pytest

from test_layer_abi import ALIAS, BASE, GB, WORKSPACE, lib, scan  # noqa: F401


def size(lib, a):  # noqa: F811
    return lib.ssm_packed_scan_workspace_size(ctypes.byref(a))


@pytest.mark.parametrize("fields", [{}, dict(chunk_len=16), dict(dstate=1), dict(tokens=20000, dim=2560, x_stride=2560, delta_stride=2560, z_stride=2560)])
def test_size_by_presence(lib, fields):  # noqa: F811
    def made(**more):
        a = scan()
        for k, v in dict(fields, **more).items():
            setattr(a, k, v)
        return a

    apart = size(lib, made())
    assert apart == size(lib, made(h_last=made().h0)) == size(lib, made(h0=BASE + 90 * GB, h_last=BASE + 90 * GB + 4)) > 0
    assert apart > size(lib, made(h0=None)) == size(lib, made(h_last=None)) > 0
    # enough for the call in place: what is refused is the alias of y behind the workspace's check
    a = made(h_last=made().h0, workspace_bytes=apart)
    a.y = a.x
    assert lib.ssm_packed_scan_fwd(ctypes.byref(a), None) == ALIAS
    a.workspace_bytes = apart - 1
    assert lib.ssm_packed_scan_fwd(ctypes.byref(a), None) == WORKSPACE
