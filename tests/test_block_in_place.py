"""Outputs in the place of inputs, at the C entry (no GPU): the same address is allowed only with the same strides, where
each element replaces itself."""
import pytest

from structured_state_space_gb300 import block
from test_block_abi import A, call, conv, lib  # noqa: F401


@pytest.mark.parametrize("kw", [dict(L=2), dict(batch=2, slots=2, y=(A, 16, 8)), dict(batch=2, slots=2, x=(A, 0, 8))])
def test_short_conv_refuses(lib, kw):  # noqa: F811
    assert call(lib, "s4_short_conv_fwd", block._CONV, *conv(**(dict(y=(A, 8, 8)) | kw))) == 1


@pytest.mark.parametrize("h_row,out_row", [(8, 16), (16, 8), (0, 8)])
def test_block_norm_refuses_a_residual_at_other_strides(lib, h_row, out_row):  # noqa: F811
    # o, gate, h, h_out, y, w_post, scale, w_pre; strides of o, gate, h, h_out, y; rows, eps, H, dtype, res_f32
    args = [A, A, 2 * A, 2 * A, 3 * A, A, A, A, 8, 8, h_row, out_row, 8, 4, 1e-5, 8, 1, 1]
    assert call(lib, "s4_block_norm_fwd", block._NORM, *args) == 1
