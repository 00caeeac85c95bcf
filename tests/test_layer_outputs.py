"""Outputs that the layer's calls make themselves are dense, whatever the strides of the
input they are like (the kernels write dense rows); checked on the CPU."""
import pytest
import torch

from selective_state_space_83_amd import layer as M


@pytest.mark.parametrize("shape,strides", [
    ((4, 8), (1, 1)), ((4, 8), (3, 1)), ((4, 8), (0, 1)), ((4, 8), (24, 1)), ((3, 5, 16), (5, 1, 1)), ((3, 5, 16), (0, 0, 1)),
    ((4, 1), (7, 3)), ((1, 8), (1, 1)), ((0, 8), (1, 1)), ((8,), (1,)),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dense(shape, strides, dtype):
    like = torch.zeros(400).as_strided(shape, strides)
    out, at = M._out(None, "y", like, like.shape, dtype, -1, torch)
    assert out.shape == like.shape and out.dtype is dtype and at == out.data_ptr()
    assert out.is_contiguous() and out.stride() == torch.empty(shape).stride()
