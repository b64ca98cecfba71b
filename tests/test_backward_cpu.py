"""The backward pass without a GPU: workspace sizes, and every refusal of the C
calls and of their Python forms before anything is launched."""
import ctypes

import pytest
import torch

from omni_modal_diffusion_b200 import build as B
from omni_modal_diffusion_b200 import h3

P = ctypes.c_void_p
# C calls: number of pointer arguments, position of `branch` among all
# arguments after dims and ranges (or None), pointers that may be NULL
CALLS = {
    "h3_adaln_norm_modulate_backward": (7, 2, {5}),
    "h3_qkv_qknorm_mrope_backward": (13, None, {9, 10, 11}),
    "h3_attention_lse": (7, None, set()),
    "h3_attention_backward": (10, None, set()),
    "h3_gated_residual_backward": (8, 4, {5, 6}),
    "h3_ffn_swiglu_backward": (10, None, {6, 7, 8}),
}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return h3.lib()


def call(lib, name, dims, ranges, pointers, branch=0):
    n, at, _ = CALLS[name]
    assert len(pointers) == n
    args = [P(p) for p in pointers]
    if at is not None:
        args.insert(at, branch)
    return getattr(lib, name)(ctypes.byref(dims) if dims else None, ctypes.byref(ranges) if ranges else None, *args,
                              None)


def good(name):
    return [16 * (i + 1) for i in range(CALLS[name][0])]


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(lib, name):
    d, r = h3.make_dims(320, 4, 896), h3.h3_make_ranges(16, 16, 32)
    n, at, optional = CALLS[name]
    assert call(lib, name, None, r, good(name)) == h3.H3_ERR_NULL
    assert call(lib, name, d, None, good(name)) == h3.H3_ERR_NULL
    for i in range(n):
        p = good(name)
        p[i] = 0
        if i not in optional and not (name == "h3_attention_lse" and i in (3, 4)):
            assert call(lib, name, d, r, p) == h3.H3_ERR_NULL, i
            assert name.encode() in lib.h3_last_error()
        p[i] = 24
        assert call(lib, name, d, r, p) == h3.H3_ERR_ALIGN, i
    if at is not None:
        assert call(lib, name, d, r, good(name), branch=2) == h3.H3_ERR_SHAPE
    assert call(lib, name, h3.make_dims(320, 4, 896, head_dim=64), r, good(name)) == h3.H3_ERR_UNSUPPORTED
    assert call(lib, name, h3.make_dims(330, 4, 896), r, good(name)) == h3.H3_ERR_UNSUPPORTED
    assert call(lib, name, h3.make_dims(320, 4, 900), r, good(name)) == h3.H3_ERR_UNSUPPORTED
    bad = h3.h3_make_ranges(16, 16, 32)
    bad.count[1] = 15
    assert call(lib, name, d, bad, good(name)) == h3.H3_ERR_SHAPE
    bad = h3.h3_make_ranges(16, 16, 32)
    bad.L_pad = 64
    assert call(lib, name, d, bad, good(name)) == h3.H3_ERR_SHAPE


def test_norm_weights_of_attention_come_together(lib):
    d, r = h3.make_dims(320, 4, 896), h3.h3_make_ranges(16, 16, 32)
    for i in (3, 4):
        p = good("h3_attention_lse")
        p[i] = 0
        assert call(lib, "h3_attention_lse", d, r, p) == h3.H3_ERR_NULL


def test_dx_must_not_be_x(lib):
    d, r = h3.make_dims(320, 4, 896), h3.h3_make_ranges(16, 16, 32)
    p = good("h3_adaln_norm_modulate_backward")
    p[4] = p[0]
    assert call(lib, "h3_adaln_norm_modulate_backward", d, r, p) == h3.H3_ERR_SHAPE


def test_workspace_bytes(lib):
    d = h3.make_dims(5376, 56, 14336)
    ops = (h3.H3_BWD_ADALN, h3.H3_BWD_QKV, h3.H3_BWD_ATTENTION, h3.H3_BWD_GATED_RESIDUAL, h3.H3_BWD_FFN)
    for op in ops:
        a, b = (h3.h3_backward_workspace_bytes(d, n, op) for n in (128, 7936))
        assert 0 < a <= b and a % 256 == 0
        assert h3.h3_backward_workspace_bytes(d, 0, op) == 0
    assert h3.h3_backward_workspace_bytes(d, 128, 5) == 0 and h3.h3_backward_workspace_bytes(d, 128, -1) == 0
    assert h3.h3_backward_workspace_bytes(d, 7936, h3.H3_BWD_ATTENTION) == 2 * 56 * 7936 * 4
    # past 32 bits: 124,032 rows of three hidden states alone are 10.7 GB
    assert h3.h3_backward_workspace_bytes(d, 124032, h3.H3_BWD_FFN) > 124032 * 3 * 14336 * 2


def test_python_forms_refuse_tensors_that_are_not_on_a_gpu(lib):
    d, r = h3.make_dims(320, 4, 896), h3.h3_make_ranges(16, 16, 32)
    f, b, w = torch.zeros(128, 320), torch.zeros(128, 320, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.uint8)
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        h3.h3_adaln_norm_modulate_backward(d, r, f, torch.zeros(3, 6, 320), h3.H3_MSA, b, f, f, None, w)
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        h3.h3_attention_backward(d, r, None, b, b, b, f, b, b, b, b, w)
