"""C-ABI contract of the residual norm's gradients from x and the residual, checked on the
CPU: what is refused (before any HIP call; the pointers are made up and never
dereferenced)."""
import ctypes

import pytest

from selective_state_space_83_amd import SSM_BF16, SSM_F32
from selective_state_space_83_amd import layer as M
from test_layer_abi import ALIAS, BASE, BIG, DTYPE, GB, NULL, OK, SHAPE, UNSUPPORTED, WORKSPACE, lib, nbwd  # noqa: F401

RES = BASE + 50 * GB
MIXED = dict(dtype=SSM_BF16, sum_dtype=SSM_F32)


@pytest.mark.parametrize("status,residual,stride,fields", [
    (NULL, None, 96, {}), (SHAPE, RES, -1, {}), (SHAPE, RES, BIG, {}), (UNSUPPORTED, RES + 2, 96, {}),
    (UNSUPPORTED, RES + 2, 96, MIXED), (ALIAS, "dx", 96, {}), (ALIAS, "dweight", 96, {}), (ALIAS, "workspace", 96, {}),
    (SHAPE, RES, 96, dict(rows=-1)), (DTYPE, RES, 96, dict(sum_dtype=SSM_BF16)), (NULL, RES, 96, dict(sum=None)),
    # x has dtype, whatever the residual's
    (WORKSPACE, RES, 96, dict(MIXED, sum=BASE + 2, workspace_bytes=4)), (UNSUPPORTED, RES, 96, dict(MIXED, sum=BASE + 1)),
], ids=lambda v: str(v))
def test_refused(lib, status, residual, stride, fields):  # noqa: F811
    a = nbwd()
    for k, v in fields.items():
        setattr(a, k, v)
    at = getattr(a, residual) if isinstance(residual, str) else residual
    assert lib.ssm_add_norm_bwd_residual(ctypes.byref(a), at, stride, None) == status, lib.ssm_last_error_message()
    assert lib.ssm_last_error_message()


def test_null_and_empty(lib):  # noqa: F811
    assert lib.ssm_add_norm_bwd_residual(None, RES, 96, None) == NULL
    assert lib.ssm_add_norm_bwd_residual(ctypes.byref(M.AddNormBwdArgs(rows=5)), None, 0, None) == OK
