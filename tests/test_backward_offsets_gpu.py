"""Attention's backward pass on keys and values that share an offset per channel.

dS sums to 0 over a row's keys, so an offset that all keys share drops out of
dQ, and one that all values share out of dP - delta, as long as every row's
delta is that of its own P and dP.  A delta that is off by e (taken from a
rounded o, say) leaves e times the mean key in dQ, which grows against the
gradient with the offsets and with the row's length.

Tolerance, in the 2-norm, in half steps of bf16 (U): P or dS rounded, the result
rounded, fp32 accumulation: 3 for dK and dV, as without offsets.  In dQ the
roundings of dS are weighted by whole keys, offset `ko` included, where the
gradient has only their spread of about 1: 1 + sqrt(1 + ko^2) half steps, and 1
for the rest.
"""
import math

import pytest
import torch

from omni_modal_diffusion_b200 import h3

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from omni_modal_diffusion_b200 import build
    build.build()
    assert torch.cuda.is_available()


def inputs(L, H, ko, vo, qo, seed):
    """q, k (normalised rows, then an offset in k's channels), v, do as
    [H][L_pad][128] bf16 with zero padding."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = h3.h3_make_ranges(0, 0, L)
    n = lambda *s: torch.empty(*s, device=DEV).normal_(generator=g)  # noqa: E731

    def heads(offset, unit):
        t = n(H, r.L_pad, 128) + offset * n(H, 1, 128)
        if unit:
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True))
        t[:, L:] = 0
        return t.to(BF16)

    return r, heads(qo, True), heads(ko, True), heads(vo, False), heads(0.0, False)


@pytest.mark.parametrize("with_norms", (True, False))
@pytest.mark.parametrize("L,H,ko,vo,qo", ((300, 2, 1, 4, 0), (1024, 2, 1, 1, 0), (1024, 1, 4, 4, 0), (1025, 2, 1, 4, 1),
                                          (4100, 1, 1, 1, 0), (129, 3, 1, 8, 1)))
def test_offsets_shared_by_all_keys_and_values(L, H, ko, vo, qo, with_norms):
    r, q, k, v, d = inputs(L, H, ko, vo, qo, L + H)
    dims = h3.make_dims(64, H, 128)
    do = d.transpose(0, 1).reshape(r.L_pad, H * 128).contiguous()
    o = torch.empty(r.L_pad, H * 128, dtype=BF16, device=DEV)
    lse = torch.empty(H, r.L_pad, dtype=F32, device=DEV)
    one = torch.ones(128, dtype=BF16, device=DEV)
    norms = {"qn_w": one, "kn_w": one} if with_norms else {}
    h3.h3_attention_lse(dims, r, q, k, v, o, lse, **norms)
    dq, dk, dv = (torch.full_like(q, math.nan) for _ in range(3))
    ws = torch.empty(h3.h3_backward_workspace_bytes(dims, r.L_pad, h3.H3_BWD_ATTENTION), dtype=torch.uint8, device=DEV)
    h3.h3_attention_backward(dims, r, q, k, v, o, lse, do, dq, dk, dv, ws)
    torch.cuda.synchronize()
    assert h3.h3_device_status() == 0
    Q, K, V, DO = (t[:, :L].double() for t in (q, k, v, d))
    c = 128 ** -0.5
    P = torch.softmax(c * Q @ K.transpose(1, 2), -1)
    dP = DO @ V.transpose(1, 2)
    dS = P * (dP - (P * dP).sum(-1, keepdim=True))
    want = {"dq": c * dS @ K, "dk": c * dS.transpose(1, 2) @ Q, "dv": P.transpose(1, 2) @ DO}
    limits = {"dq": 2 + math.sqrt(1 + ko * ko), "dk": 3, "dv": 3}
    for (name, w), got in zip(want.items(), (dq, dk, dv)):
        off = float((got[:, :L].double() - w).norm() / w.norm())
        assert off <= limits[name] * U, f"{name}: {off:.2e}"
        assert torch.all(got[:, L:] == 0)
