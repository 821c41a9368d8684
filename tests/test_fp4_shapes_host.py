"""Sizes of 4-bit buffers that there are none of: the library's error, before anything else."""

import pytest

import tenant_serving_b200 as bd


@pytest.mark.parametrize("rows,cols,fmt", [(0, 64, bd.BD_FP4_NV), (4, 48, bd.BD_FP4_NV), (4, 64, 2), (-1, 64, bd.BD_FP4_MX)])
def test_shapes_of_no_matrix(rows, cols, fmt):
    for call in (lambda: bd.fp4_scales_shape(rows, cols, fmt), lambda: bd.fp4_buffers(rows, cols, fmt, "cpu")):
        with pytest.raises(bd.BitDeltaError) as e:
            call()
        assert e.value.code == bd.BD_ERR_SHAPE
