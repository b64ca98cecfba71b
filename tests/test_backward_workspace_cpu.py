"""Workspace sizes of the backward calls for arguments that the calls refuse."""
import pytest

from omni_modal_diffusion_b200 import build as B
from omni_modal_diffusion_b200 import h3

OPS = (h3.H3_BWD_ADALN, h3.H3_BWD_QKV, h3.H3_BWD_ATTENTION, h3.H3_BWD_GATED_RESIDUAL, h3.H3_BWD_FFN)


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


@pytest.mark.parametrize("op", OPS)
def test_sizes_of_refused_arguments_are_zero(op):
    good = h3.make_dims(320, 4, 896)
    assert h3.h3_backward_workspace_bytes(good, 256, op) > 0
    for rows in (-128, 0, 1, 100, 130):
        assert h3.h3_backward_workspace_bytes(good, rows, op) == 0, rows
    split = h3.make_dims(320, 4, 896)
    split.I = 256
    for dims in (h3.make_dims(330, 4, 896), h3.make_dims(8256, 4, 896), h3.make_dims(0, 4, 896), h3.make_dims(320, 0, 896),
                 h3.make_dims(320, 4, 900), h3.make_dims(320, 4, 896, head_dim=64), split):
        assert h3.h3_backward_workspace_bytes(dims, 256, op) == 0
