"""GPU tests of the block's backward pass against the float64 oracle.

Tolerances: every element within the oracle's bound for it (half a bf16 step
for each operand and result that is rounded, carried through sums of absolute
values, plus fp32 accumulation), which holds whatever the signs; and for random
inputs the error's 2-norm within ROUNDINGS half steps of the result's, one for
each rounding on the way to it (independent errors add in squares, so this is
not reached either).
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import h3_oracle as O
from oracle import h3_oracle_bwd as G
from omni_modal_diffusion_b200 import h3
from omni_modal_diffusion_b200 import synthetic as S
from omni_modal_diffusion_b200.pipeline import H3BlockTrain, to_dev_bf16

from parity_util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from omni_modal_diffusion_b200 import build
    build.build()
    assert torch.cuda.is_available()


def inside(got, want, name, roundings=None, norm=True):
    ref, bound = want
    got = to_np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), name
    off = np.abs(got - ref)
    worst = off - bound - 1e-30
    assert np.all(worst <= 0), f"{name}: {off.flat[worst.argmax()]:.3e} off at {worst.argmax()}, bound {bound.flat[worst.argmax()]:.3e}"
    if norm and roundings:
        scale = np.linalg.norm(ref)
        assert np.linalg.norm(off) <= roundings * U * scale, f"{name}: {np.linalg.norm(off) / scale:.2e}"


class Inputs:
    """Seeded inputs of one set of sizes; `b`, `f`: as bf16 and fp32 CUDA
    tensors with the padding rows filled with `fill`."""

    def __init__(self, counts, D=320, H=2, F=256, seed=0, pad_tiles=0, fill=float("nan")):
        self.rng = np.random.default_rng(seed)
        self.D, self.H, self.F, self.I = D, H, F, 128 * H
        self.dims = h3.make_dims(D, H, F)
        self.ranges = h3.h3_make_ranges(*counts)
        self.ranges.L_pad += 128 * pad_tiles
        self.r = O.pack_ranges(*counts)
        self.L, self.Lp, self.fill = self.r["L"], self.ranges.L_pad, fill

    def normal(self, *shape, std=1.0, mean=0.0, bf16=True):
        a = self.rng.standard_normal(shape, dtype=np.float32) * np.float32(std) + np.float32(mean)
        return S.bf16_round(a) if bf16 else a

    def rows(self, a, dtype=BF16, axis=0):
        """Token rows padded to L_pad."""
        pad = [(0, 0)] * a.ndim
        pad[axis] = (0, self.Lp - self.L)
        return torch.from_numpy(np.pad(a.astype(np.float32), pad, constant_values=self.fill)).to(DEV).to(dtype)

    def heads(self, a):
        """[L, H, 128] -> [H, L_pad, 128]"""
        return self.rows(np.ascontiguousarray(a.transpose(1, 0, 2)), axis=1)

    def ws(self, op):
        return torch.empty(h3.h3_backward_workspace_bytes(self.dims, self.Lp, op), dtype=torch.uint8, device=DEV).fill_(255)

    def empty(self, *shape, dtype=BF16):
        return torch.full(shape, float("nan"), dtype=dtype, device=DEV)

    def finish(self):
        torch.cuda.synchronize()
        assert h3.h3_device_status() == 0


def dev(a, dtype=BF16):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)


# token counts (text, audio, video): one token, tile edges, empty modalities, ragged tails
COUNTS = [(1, 0, 0), (0, 0, 1), (1, 1, 1), (127, 0, 0), (0, 128, 0), (0, 1, 128), (37, 58, 240), (256, 3, 126),
          (5, 0, 252)]
WIDTHS = [(64, 1, 128), (320, 3, 384), (576, 6, 1280)]


def sizes():
    out = [(c, WIDTHS[i % 3], 0) for i, c in enumerate(COUNTS)]
    out += [((130, 0, 1), WIDTHS[0], 1), ((37, 58, 33), WIDTHS[1], 2)]  # rows padded by whole tiles
    return out


SIZES = pytest.mark.parametrize("counts,widths,pad", sizes(), ids=lambda v: str(v).replace(" ", ""))


# ---------------------------------------------------------------- AdaLN

def run_adaln(t, branch, x, mod, dy, dres, in_place=False):
    dmod = t.empty(3, 6, t.D)
    res = t.rows(dres, F32)
    dx = res if in_place else t.empty(t.Lp, t.D, dtype=F32)
    h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, t.rows(x, F32), dev(mod, F32), branch, t.rows(dy), res, dx,
                                       dmod, t.ws(h3.H3_BWD_ADALN))
    t.finish()
    return dx, dmod


def check_adaln(t, branch, x, mod, dy, dres, **kw):
    dx, dmod = run_adaln(t, branch, x, mod, dy, dres, **kw)
    want = G.adaln_modulate(x, mod, t.r, branch, dy, dres, err=True)
    inside(dx[:t.L], want[0], "dx")
    assert torch.all(dx[t.L:] == 0)
    b = 3 * branch
    inside(dmod[:, b], want[1], "dshift")
    inside(dmod[:, b + 1], want[2], "dscale")
    others = [i for i in range(6) if i not in (b, b + 1)]
    assert torch.all(torch.isnan(dmod[:, others].float()))  # the other slots are left as they were


@SIZES
@pytest.mark.parametrize("branch", (h3.H3_MSA, h3.H3_MLP))
def test_adaln(counts, widths, pad, branch):
    t = Inputs(counts, *widths, seed=branch, pad_tiles=pad)
    check_adaln(t, branch, t.normal(t.L, t.D, std=3.0, mean=0.5, bf16=False), t.normal(3, 6, t.D, std=0.1, bf16=False),
                t.normal(t.L, t.D, std=1e-3), t.normal(t.L, t.D, std=1e-3, bf16=False), in_place=branch == h3.H3_MLP)


@pytest.mark.parametrize("D", (64, 1024, 1088, 2048, 2112, 4096, 5376, 6208, 7232, 8192))
def test_adaln_every_width_class(D):
    t = Inputs((3, 300, 9), D, 1, 128, seed=D)
    check_adaln(t, 0, t.normal(t.L, D, bf16=False), t.normal(3, 6, D, std=0.1, bf16=False), t.normal(t.L, D),
                t.normal(t.L, D, bf16=False))


def test_adaln_rows_far_from_zero_and_nearly_constant():
    """Mean 100 times the spread: the variance is not taken as a difference of
    squares.  A constant row (variance 0) stays finite."""
    t = Inputs((40, 0, 30), 320, seed=3)
    x = t.normal(t.L, t.D, mean=100.0, bf16=False)
    check_adaln(t, 1, x, t.normal(3, 6, t.D, std=0.1, bf16=False), t.normal(t.L, t.D), t.normal(t.L, t.D, bf16=False))
    dx, dmod = run_adaln(t, 1, np.full((t.L, t.D), 2.0, np.float32), np.zeros((3, 6, t.D)), t.normal(t.L, t.D),
                         np.zeros((t.L, t.D)))
    assert torch.all(torch.isfinite(dx)) and torch.all(dmod[:, 4] == 0)


def test_adaln_many_rows():
    """More rows than CTAs: every CTA sums a run of rows."""
    t = Inputs((700, 1, 2500), 128, seed=5)
    check_adaln(t, 0, t.normal(t.L, t.D, bf16=False), t.normal(3, 6, t.D, std=0.1, bf16=False), t.normal(t.L, t.D),
                t.normal(t.L, t.D, bf16=False))


# ---------------------------------------------------------------- QKV

@SIZES
def test_qkv(counts, widths, pad):
    D, H, F = widths
    t = Inputs(counts, D, H, F, seed=11, pad_tiles=pad)
    xm, W = t.normal(t.L, D), t.normal(3 * t.I, D, std=0.05)
    qn, kn = t.normal(128, std=0.1, mean=1.0), t.normal(128, std=0.1, mean=1.0)
    pos = t.rng.integers(0, 90, (t.L, 3)).astype(np.float32)
    ds = [t.normal(t.L, H, 128, std=s) for s in (1e-3, 1e-2, 1.0)]
    out = [t.empty(t.Lp, D), t.empty(3 * t.I, D), t.empty(128), t.empty(128)]
    h3.h3_qkv_qknorm_mrope_backward(t.dims, t.ranges, t.rows(xm), dev(W), dev(qn), dev(kn), t.rows(pos, F32),
                                    *(t.heads(d) for d in ds), *out, t.ws(h3.H3_BWD_QKV))
    t.finish()
    want = G.qkv_qknorm_mrope(xm, W, qn, kn, pos, H, *ds, err=True)
    inside(out[0][:t.L], want[0], "dxm", 2)
    assert torch.all(out[0][t.L:] == 0)
    for got, w, name, n in zip(out[1:], want[1:], ("dWqkv", "dqn_w", "dkn_w"), (2, 1.1, 1.1)):
        inside(got, w, name, n)


# ---------------------------------------------------------------- attention

def run_attention(t, q, k, v, do, qn=None, kn=None):
    """(o, lse, dq, dk, dv) of one training pass."""
    gq, gk, gv, gdo = t.heads(q), t.heads(k), t.heads(v), t.rows(do.reshape(t.L, -1))
    for g in (gq, gk, gv):  # the forward call wants finite padding, as the QKV call leaves it
        g[:, t.L:] = 0
    o, lse = t.empty(t.Lp, t.I), t.empty(t.H, t.Lp, dtype=F32)
    norms = {} if qn is None else {"qn_w": dev(qn), "kn_w": dev(kn)}
    h3.h3_attention_lse(t.dims, t.ranges, gq, gk, gv, o, lse, **norms)
    again = t.empty(t.Lp, t.I)
    h3.h3_attention(t.dims, t.ranges, gq, gk, gv, again, **norms)
    assert torch.equal(o, again)
    assert torch.all(lse[:, t.L:] == 0) and torch.all(o[t.L:] == 0)
    for g in (gq, gk, gv):  # the backward call reads no padding
        g[:, t.L:] = t.fill
    o[t.L:], lse[:, t.L:] = t.fill, t.fill
    grads = [t.empty(t.H, t.Lp, 128) for _ in range(3)]
    h3.h3_attention_backward(t.dims, t.ranges, gq, gk, gv, o, lse, gdo, *grads, t.ws(h3.H3_BWD_ATTENTION))
    t.finish()
    return o, lse, *grads


def check_attention(t, q, k, v, do, norm=True, **kw):
    o, lse, *grads = run_attention(t, q, k, v, do, **kw)
    ref = G.attention_lse(q, k)
    # scores are sums of 128 exact products in fp32 and the exponent scale one more rounding
    slack = 2.0 ** -20 * (1.0 + np.abs(ref).max() + np.einsum("ihd,jhd->hij", np.abs(q), np.abs(k)).max() / 11.3)
    assert np.abs(to_np(lse)[:, :t.L] - ref).max() <= slack
    for g, want, name in zip(grads, G.attention(q, k, v, do, err=True), ("dq", "dk", "dv")):
        inside(to_np(g)[:, :t.L].transpose(1, 0, 2), want, name, 3, norm=norm)
        assert torch.all(g[:, t.L:] == 0)


def normalised(t, w):
    x = t.normal(t.L, t.H, 128, bf16=False).astype(np.float64)
    return S.bf16_round((x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w).astype(np.float32))


@SIZES
@pytest.mark.parametrize("with_norms", (True, False))
def test_attention(counts, widths, pad, with_norms):
    t = Inputs(counts, *widths, seed=21, pad_tiles=pad)
    qn, kn = t.normal(128, std=0.1, mean=1.0), t.normal(128, std=0.1, mean=1.0)
    q, k = normalised(t, qn), normalised(t, kn)
    # one token: dq and dk are 0 up to o's rounding, so their own norm says nothing
    check_attention(t, q, k, t.normal(t.L, t.H, 128), t.normal(t.L, t.H, 128, std=1e-2), norm=t.L > 1,
                    **({"qn": qn, "kn": kn} if with_norms else {}))


@pytest.mark.parametrize("L", (383, 512, 641, 1025))
def test_attention_several_tiles(L):
    t = Inputs((L // 3, 0, L - L // 3), 64, 3, 128, seed=L)
    one = np.ones(128, np.float32)
    check_attention(t, normalised(t, one), normalised(t, one), t.normal(t.L, t.H, 128), t.normal(t.L, t.H, 128),
                    qn=one, kn=one)


@pytest.mark.parametrize("scale", (0.0, 3.0, 12.0))
def test_attention_flat_and_peaked_rows(scale):
    """Norm weights of 0 (uniform rows), 3 (scores to +-100: past the forward
    call's static bound, which then recomputes) and 12 (one-hot rows, scores to
    +-1600)."""
    t = Inputs((100, 0, 170), 64, 2, 128, seed=31)
    qn, kn = np.full(128, scale, np.float32), np.ones(128, np.float32) * max(scale, 1.0)
    q, k = normalised(t, qn), normalised(t, kn)
    # k rows repeated over the queries' own positions give every row a dominant key
    check_attention(t, q, S.bf16_round((q if scale == 12.0 else k).astype(np.float32)), t.normal(t.L, t.H, 128),
                    t.normal(t.L, t.H, 128), norm=False, qn=qn, kn=kn)


def test_attention_shared_gradient_of_equal_keys():
    """All keys and values equal: P is uniform, dq is 0 up to rounding, and dk,
    dv are the same for every key."""
    t = Inputs((0, 0, 200), 64, 1, 128, seed=41)
    k, v = (np.repeat(t.normal(1, 1, 128), t.L, axis=0) for _ in range(2))
    check_attention(t, t.normal(t.L, 1, 128), k, v, t.normal(t.L, 1, 128), norm=False)


# ---------------------------------------------------------------- gated out-projection, feed-forward

def mod_with_zero_gates(t):
    """Modulation whose audio gates are all 0 and some others too (blocks start
    from zero gates)."""
    mod = t.normal(3, 6, t.D, std=0.3, bf16=False)
    mod[1, [2, 5]] = 0
    mod[:, [2, 5], ::7] = 0
    return mod


@SIZES
@pytest.mark.parametrize("branch", (h3.H3_MSA, h3.H3_MLP))
def test_gated_residual(counts, widths, pad, branch):
    D, H, F = widths
    t = Inputs(counts, D, H, F, seed=51, pad_tiles=pad)
    dx, o, Wo, mod = t.normal(t.L, D, bf16=False), t.normal(t.L, t.I), t.normal(D, t.I, std=0.05), mod_with_zero_gates(t)
    do, dWo, dmod = t.empty(t.Lp, t.I), t.empty(D, t.I), t.empty(3, 6, D)
    h3.h3_gated_residual_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(o), dev(Wo), dev(mod, F32), do, dWo, dmod,
                                  t.ws(h3.H3_BWD_GATED_RESIDUAL), branch=branch)
    t.finish()
    want = G.gated_residual(dx, o, Wo, mod, t.r, branch=branch, err=True)
    inside(do[:t.L], want[0], "do", 2)
    assert torch.all(do[t.L:] == 0)
    inside(dWo, want[1], "dWo", 2)
    slot = 3 * branch + 2
    inside(dmod[:, slot], want[2], "dgate", 2)
    assert torch.all(torch.isnan(dmod[:, [i for i in range(6) if i != slot]].float()))


@SIZES
def test_ffn(counts, widths, pad):
    D, H, F = widths
    t = Inputs(counts, D, H, F, seed=61, pad_tiles=pad)
    dx, xm, mod = t.normal(t.L, D, bf16=False), t.normal(t.L, D), mod_with_zero_gates(t)
    Wgu, Wd = t.normal(2 * F, D, std=0.1), t.normal(D, F, std=0.05)
    dxm, dWgu, dWd, dmod = t.empty(t.Lp, D), t.empty(2 * F, D), t.empty(D, F), t.empty(3, 6, D)
    h3.h3_ffn_swiglu_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(xm), dev(Wgu), dev(Wd), dev(mod, F32), dxm,
                              dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
    t.finish()
    want = G.ffn_swiglu(dx, xm, Wgu, Wd, mod, t.r, err=True)
    inside(dxm[:t.L], want[0], "dxm", 3)
    assert torch.all(dxm[t.L:] == 0)
    inside(dWgu, want[1], "dWgu", 3)
    inside(dWd, want[2], "dWd", 3)
    inside(dmod[:, 5], want[3], "dgate", 3)
    assert torch.all(torch.isnan(dmod[:, :5].float()))


def test_ffn_saturated_gates():
    """Gate pre-activations to +-400: exp overflows on one side, SiLU and its
    derivative reach their limits, nothing is NaN."""
    t = Inputs((20, 0, 40), 64, 1, 128, seed=71)
    dx, xm, mod = t.normal(t.L, 64, bf16=False), t.normal(t.L, 64), t.normal(3, 6, 64, bf16=False)
    Wgu, Wd = t.normal(256, 64, std=12.0), t.normal(64, 128, std=0.05)
    dxm, dWgu, dWd, dmod = t.empty(t.Lp, 64), t.empty(256, 64), t.empty(64, 128), t.empty(3, 6, 64)
    h3.h3_ffn_swiglu_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(xm), dev(Wgu), dev(Wd), dev(mod, F32), dxm,
                              dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
    t.finish()
    with np.errstate(over="ignore"):
        want = G.ffn_swiglu(dx, xm, Wgu, Wd, mod, t.r, err=True)
    for got, w, name in zip((dxm[:t.L], dWgu, dWd, dmod[:, 5]), want, ("dxm", "dWgu", "dWd", "dgate")):
        inside(got, w, name)


@pytest.mark.parametrize("counts,widths", (((40, 0, 260), (1024, 16, 4096)), ((100, 33, 200), (2048, 16, 2048)),
                                           ((0, 513, 7), (1984, 15, 1920))), ids=str)
def test_products_over_several_turns(counts, widths):
    """More output tiles than the GPU has CTA pairs, in one launch: pairs that
    the first product's last turn leaves out go on with the next product's."""
    test_qkv(counts, widths, 0)
    test_gated_residual(counts, widths, 0, h3.H3_MSA)
    test_ffn(counts, widths, 1)


# ---------------------------------------------------------------- long sequences

LONG = (512, 1200, 122304)  # the packed 15 s sequence: 124,016 tokens


def test_attention_long():
    """One head over 124,016 tokens: dq of sampled queries and dk, dv of sampled
    keys (the last ones of the ragged tile among them) against float64 on the
    GPU, lse of every row."""
    t = Inputs(LONG, 64, 1, 128, seed=111, fill=0.0)
    L = t.L
    g = torch.Generator(device=DEV)
    g.manual_seed(111)
    draw = lambda std: torch.empty(1, t.Lp, 128, device=DEV).normal_(0, std, generator=g)  # noqa: E731
    unit = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True))  # noqa: E731
    q, k, v, do = (x.to(BF16) for x in (unit(draw(1.0)), unit(draw(1.0)), draw(1.0), draw(1e-2)))
    for x in (q, k, v, do):
        x[:, L:] = 0
    one = torch.ones(128, dtype=BF16, device=DEV)
    o, lse, do = t.empty(t.Lp, 128), t.empty(1, t.Lp, dtype=F32), do.view(t.Lp, 128)
    h3.h3_attention_lse(t.dims, t.ranges, q, k, v, o, lse, qn_w=one, kn_w=one)
    dq, dk, dv = (t.empty(1, t.Lp, 128) for _ in range(3))
    h3.h3_attention_backward(t.dims, t.ranges, q, k, v, o, lse, do, dq, dk, dv, t.ws(h3.H3_BWD_ATTENTION))
    t.finish()
    Q, K, V, DO = (x.view(t.Lp, 128)[:L].double() for x in (q, k, v, do))
    c = 128 ** -0.5
    ref_lse, O_ = [], []
    for i in range(0, L, 4096):
        s = c * (Q[i:i + 4096] @ K.T)
        ref_lse.append(torch.logsumexp(s, 1))
        O_.append(torch.exp(s - ref_lse[-1][:, None]) @ V)
    ref_lse, O_ = torch.cat(ref_lse), torch.cat(O_)
    # fp32 sums of 124,016 exponentials of scores below 12
    assert (lse[0, :L].double() - ref_lse).abs().max() <= 2.0 ** -16
    delta = (DO * O_).sum(1)
    rows = torch.cat((torch.arange(0, L, L // 61, device=DEV), torch.arange(L - 5, L, device=DEV)))
    p = torch.exp(c * (Q[rows] @ K.T) - ref_lse[rows, None])
    want = c * ((p * (DO[rows] @ V.T - delta[rows, None])) @ K)
    pk = torch.exp(c * (Q @ K[rows].T) - ref_lse[:, None])
    want_dv = pk.T @ DO
    want_dk = c * ((pk * (DO @ V[rows].T - delta[:, None])).T @ Q)
    for name, got, ref in (("dq", dq, want), ("dk", dk, want_dk), ("dv", dv, want_dv)):
        off = (got[0, rows].double() - ref).norm() / ref.norm()
        assert off <= 3 * U, (name, float(off))  # P, dS and o, and the result: three roundings each
        assert torch.all(got[0, L:] == 0)


def test_products_long():
    """124,016 tokens through narrow layers: contractions over the tokens in
    splits."""
    t = Inputs(LONG, 64, 1, 128, seed=121)
    dx, xm, mod = t.normal(t.L, 64, bf16=False), t.normal(t.L, 64), mod_with_zero_gates(t)
    Wgu, Wd = t.normal(256, 64, std=0.2), t.normal(64, 128, std=0.1)
    dxm, dWgu, dWd, dmod = t.empty(t.Lp, 64), t.empty(256, 64), t.empty(64, 128), t.empty(3, 6, 64)
    h3.h3_ffn_swiglu_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(xm), dev(Wgu), dev(Wd), dev(mod, F32), dxm,
                              dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
    t.finish()
    want = G.ffn_swiglu(dx, xm, Wgu, Wd, mod, t.r, err=True)
    for got, w, name in zip((dxm[:t.L], dWgu, dWd, dmod[:, 5]), want, ("dxm", "dWgu", "dWd", "dgate")):
        inside(got, w, name, 3)
    check_adaln(t, 0, t.normal(t.L, 64, std=3.0, bf16=False), t.normal(3, 6, 64, std=0.1, bf16=False),
                t.normal(t.L, 64), t.normal(t.L, 64, bf16=False))


def test_gated_residual_wide_and_long():
    """124,016 tokens at full width, where byte offsets pass 2^31: sampled rows
    of do, and of dWo and the gate sampled channels, against float64 on the GPU."""
    t = Inputs(LONG, 5376, 56, 128, seed=131, fill=0.0)
    L, D, I = t.L, t.D, t.I
    g = torch.Generator(device=DEV)
    g.manual_seed(131)
    normal = lambda *s, std=1.0, dt=BF16: torch.empty(*s, device=DEV, dtype=dt).normal_(0, std, generator=g)  # noqa: E731
    dx, o, Wo, mod = normal(t.Lp, D, dt=F32), normal(t.Lp, I), normal(D, I, std=0.02), normal(3, 6, D, dt=F32)
    do, dWo, dmod = t.empty(t.Lp, I), t.empty(D, I), t.empty(3, 6, D)
    h3.h3_gated_residual_backward(t.dims, t.ranges, dx, o, Wo, mod, do, dWo, dmod, t.ws(h3.H3_BWD_GATED_RESIDUAL))
    t.finish()
    gate = torch.repeat_interleave(mod[:, 2], torch.tensor(LONG, device=DEV), dim=0)
    rows = torch.cat((torch.arange(0, L, 4001, device=DEV), torch.arange(L - 3, L, device=DEV)))
    ref = (dx[rows] * gate[rows]).double() @ Wo.double()
    assert (do[rows].double() - ref).norm() <= 2 * U * ref.norm()
    assert torch.all(do[L:] == 0)
    ch = torch.tensor([0, 1, 127, 128, 2500, D - 1], device=DEV)
    dW = torch.zeros(len(ch), I, device=DEV, dtype=torch.float64)
    G_ = torch.zeros(3, len(ch), I, device=DEV, dtype=torch.float64)
    for m, (a, n) in enumerate(zip((0, 512, 1712), LONG)):
        for i in range(a, a + n, 8192):
            e = min(i + 8192, a + n)
            G_[m] += dx[i:e, ch].double().T @ o[i:e].double()
        dW += mod[m, 2, ch].double()[:, None] * G_[m]
    assert (dWo[ch].double() - dW).norm() <= 2 * U * dW.norm()
    dg = (G_ * Wo[ch].double()).sum(2)
    assert (dmod[:, 2, ch].double() - dg).norm() <= 2 * U * dg.norm()


# ---------------------------------------------------------------- frozen weights

def test_gradients_that_are_not_wanted_are_not_written():
    """Every subset of the optional outputs: those asked for are the same bits
    as with all of them."""
    D, H, F = 320, 3, 384
    t = Inputs((37, 5, 90), D, H, F, seed=81, fill=0.0)
    r, d = t.ranges, t.dims
    dx, xm, mod = t.rows(t.normal(t.L, D, bf16=False), F32), t.rows(t.normal(t.L, D)), dev(mod_with_zero_gates(t), F32)
    Wgu, Wd, Wo = dev(t.normal(2 * F, D, std=0.1)), dev(t.normal(D, F, std=0.05)), dev(t.normal(D, t.I, std=0.05))
    W, qn, kn = dev(t.normal(3 * t.I, D, std=0.05)), dev(t.normal(128, mean=1.0)), dev(t.normal(128, mean=1.0))
    pos, o = t.rows(t.rng.integers(0, 9, (t.L, 3)).astype(np.float32), F32), t.rows(t.normal(t.L, t.I))
    ds = [t.heads(t.normal(t.L, H, 128)) for _ in range(3)]

    def ffn(dWgu, dWd, dmod):
        out = t.empty(t.Lp, D)
        h3.h3_ffn_swiglu_backward(d, r, dx, xm, Wgu, Wd, mod, out, dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
        return out

    def gated(dWo, dmod):
        out = t.empty(t.Lp, t.I)
        h3.h3_gated_residual_backward(d, r, dx, o, Wo, mod, out, dWo, dmod, t.ws(h3.H3_BWD_GATED_RESIDUAL))
        return out

    def qkv(dW, dqn, dkn):
        out = t.empty(t.Lp, D)
        h3.h3_qkv_qknorm_mrope_backward(d, r, xm, W, qn, kn, pos, *ds, out, dW, dqn, dkn, t.ws(h3.H3_BWD_QKV))
        return out

    def adaln(dmod):
        out = t.empty(t.Lp, D, dtype=F32)
        h3.h3_adaln_norm_modulate_backward(d, r, dx, mod, 0, xm, dx, out, dmod, t.ws(h3.H3_BWD_ADALN))
        return out

    for f, shapes in ((ffn, ((2 * F, D), (D, F), (3, 6, D))), (gated, ((D, t.I), (3, 6, D))),
                      (qkv, ((3 * t.I, D), (128,), (128,))), (adaln, ((3, 6, D),))):
        full = [t.empty(*s).zero_() for s in shapes]
        main = f(*full)
        for wanted in itertools.product((False, True), repeat=len(shapes)):
            some = [torch.zeros_like(a) if w else None for a, w in zip(full, wanted)]
            assert torch.equal(f(*some), main)
            assert all(s is None or torch.equal(s, a) for s, a in zip(some, full)), (f.__name__, wanted)
    t.finish()


# ---------------------------------------------------------------- a whole block

TINY = dict(counts=(37, 58, 240), D=320, H=4, F=896)


def block_inputs(seed, counts, D, H, F):
    t = Inputs(counts, D, H, F, seed=seed, fill=0.0)
    W = {"Wqkv": t.normal(3 * t.I, D, std=0.05), "qn_w": t.normal(128, std=0.1, mean=1.0),
         "kn_w": t.normal(128, std=0.1, mean=1.0), "Wo": t.normal(D, t.I, std=0.05), "Wgu": t.normal(2 * F, D, std=0.05),
         "Wd": t.normal(D, F, std=0.05)}
    x, mod, dx = t.normal(t.L, D, bf16=False), t.normal(3, 6, D, std=0.3, bf16=False), t.normal(t.L, D, std=1e-2, bf16=False)
    pos = t.rng.integers(0, 20, (t.L, 3)).astype(np.float32)
    return t, W, x, mod, dx, pos


def test_block_backward_through_its_own_path():
    """Forward and backward of a whole block as a training step runs them,
    against the oracle's chain and against differences of the oracle's forward
    pass.  Every gradient has passed at most 12 roundings to bf16 (xm, q/k/v, P,
    o, dxm, dgu, ... on both passes): 2-norm within 12 half steps."""
    t, W, x, mod, dx, pos = block_inputs(91, **TINY)
    d = {n: dev(w) for n, w in W.items()}
    tr = H3BlockTrain(t.dims, t.ranges)
    gx, gmod, gpos, gdx = t.rows(x, F32), dev(mod, F32), t.rows(pos, F32), t.rows(dx, F32)
    tr.forward(gx, gmod, gpos, d)
    g = tr.backward(gdx, gmod, gpos, d)
    t.finish()
    args = [W[n] for n in ("Wqkv", "qn_w", "kn_w", "Wo", "Wgu", "Wd")]
    y = O.block_forward(x, mod, t.r, pos, *args, t.H)
    assert np.abs(to_np(gx)[:t.L] - y).max() <= 3e-2 * np.sqrt((y * y).mean())
    ref_dx, ref = G.block(x, mod, t.r, pos, *args, t.H, dx)
    for name, got, want in [("dx", to_np(gdx)[:t.L], ref_dx)] + [(n, to_np(g[n]), ref[n]) for n in g]:
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off <= 12 * U, (name, off)
    assert torch.all(gdx[t.L:] == 0)
    # along a random direction of x and of each weight
    rng = np.random.default_rng(92)
    for name in ("x", "Wqkv", "Wd", "mod"):
        a = {"x": x, "mod": mod, **W}[name].astype(np.float64)
        v = rng.standard_normal(a.shape) * np.sqrt((a * a).mean())
        eps = 1e-4

        def loss(s):
            p = {"x": x, "mod": mod, **W, name: a + s * v}
            return float((O.block_forward(p["x"], p["mod"], t.r, pos, *[p[n] for n in W], t.H) * dx).sum())

        num = (loss(eps) - loss(-eps)) / (2 * eps)
        got = to_np(gdx)[:t.L] if name == "x" else to_np(g[name])
        # the gradient's error in a random direction: its 2-norm's share, with
        # a factor of 4 for the direction's own spread
        assert abs(float((got * v).sum()) - num) <= 4 * 12 * U * np.linalg.norm(got) * np.sqrt((v * v).mean()), name


def test_block_backward_frozen_weights_and_repeat():
    """A frozen block gives the same dx, and the same call the same bits."""
    t, W, x, mod, dx, pos = block_inputs(95, **TINY)
    d = {n: dev(w) for n, w in W.items()}
    tr = H3BlockTrain(t.dims, t.ranges)
    gmod, gpos = dev(mod, F32), t.rows(pos, F32)
    outs = []
    for frozen in ((), (), H3BlockTrain.WEIGHTS + ("mod",)):
        tr.forward(t.rows(x, F32), gmod, gpos, d)
        gdx = t.rows(dx, F32)
        outs.append((gdx, tr.backward(gdx, gmod, gpos, d, frozen=frozen)))
    t.finish()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][0], outs[2][0])
    assert all(torch.equal(outs[0][1][n], outs[1][1][n]) for n in outs[0][1]) and outs[2][1] == {}
    with pytest.raises(ValueError, match="unknown names"):
        tr.backward(outs[0][0], gmod, gpos, d, frozen=("W",))


def test_block_backward_captured_and_replayed_on_another_stream():
    """Forward and backward captured into a graph on a side stream, replayed on
    new inputs in the captured buffers: the eager run's bits."""
    t, W, x, mod, dx, pos = block_inputs(97, **TINY)
    d = {n: dev(w) for n, w in W.items()}
    gmod, gpos = dev(mod, F32), t.rows(pos, F32)
    tr = H3BlockTrain(t.dims, t.ranges)
    sx, sdx = torch.zeros(t.Lp, t.D, device=DEV), torch.zeros(t.Lp, t.D, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # warm-up: function attributes are set before the capture
        tr.forward(sx, gmod, gpos, d)
        tr.backward(sdx, gmod, gpos, d)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tr.forward(sx, gmod, gpos, d)
        g = tr.backward(sdx, gmod, gpos, d)
    for seed in (1, 2):
        t.rng = np.random.default_rng(seed)
        nx, ndx = t.rows(t.normal(t.L, t.D, bf16=False), F32), t.rows(t.normal(t.L, t.D, bf16=False), F32)
        sx.copy_(nx)
        sdx.copy_(ndx)
        graph.replay()
        torch.cuda.synchronize()
        other = H3BlockTrain(t.dims, t.ranges)
        ex, edx = nx.clone(), ndx.clone()
        other.forward(ex, gmod, gpos, d)
        want = other.backward(edx, gmod, gpos, d)
        t.finish()
        assert torch.equal(sx, ex) and torch.equal(sdx, edx)
        assert all(torch.equal(g[n], want[n]) for n in want)


def test_two_streams_at_once():
    """Two blocks with their own buffers on two streams give what each gives
    alone."""
    jobs = []
    for seed in (101, 102):
        t, W, x, mod, dx, pos = block_inputs(seed, **TINY)
        d = {n: dev(w) for n, w in W.items()}
        jobs.append((t, d, x, dev(mod, F32), dx, t.rows(pos, F32), H3BlockTrain(t.dims, t.ranges)))

    def run(job, stream):
        t, d, x, mod, dx, pos, tr = job
        gx, gdx = t.rows(x, F32), t.rows(dx, F32)
        torch.cuda.synchronize()
        return gx, gdx, lambda: (tr.forward(gx, mod, pos, d, stream=stream), tr.backward(gdx, mod, pos, d, stream=stream))[1]

    alone = []
    for job in jobs:
        gx, gdx, go = run(job, None)
        g = go()
        job[0].finish()
        alone.append((gx, gdx, g))
    s = [torch.cuda.Stream() for _ in jobs]
    both = [run(job, st) for job, st in zip(jobs, s)]
    grads = [go() for _, _, go in both]
    torch.cuda.synchronize()
    for (gx, gdx, _), g, (ax, adx, ag) in zip(both, grads, alone):
        assert torch.equal(gx, ax) and torch.equal(gdx, adx) and all(torch.equal(g[n], ag[n]) for n in ag)


def test_captured_behind_copies_memsets_and_another_stream():
    """Each call captured right behind a memory copy, a memset and a join with
    a second stream that fills its inputs: replays give the eager call's bits
    (no kernel of a chain starts on inputs that are not there yet)."""
    t = Inputs((37, 58, 1900), 576, 6, 1280, seed=113, fill=0.0)
    mod, pos = dev(t.normal(3, 6, t.D, std=0.3), F32), t.rows(t.rng.integers(0, 20, (t.L, 3)), F32)
    W = {n: dev(t.normal(*s, std=0.05)) for n, s in (("qkv", (3 * t.I, t.D)), ("o", (t.D, t.I)), ("gu", (2 * t.F, t.D)),
                                                     ("d", (t.D, t.F)))}
    w = dev(t.normal(128, std=0.1, mean=1.0))
    src = {n: f(t.normal(*s)) for n, s, f in (
        ("xm", (t.L, t.D), t.rows), ("o", (t.L, t.I), t.rows), ("do", (t.L, t.I), t.rows),
        ("q", (t.L, t.H, 128), t.heads), ("k", (t.L, t.H, 128), t.heads), ("v", (t.L, t.H, 128), t.heads))}
    src |= {n: t.rows(t.normal(t.L, t.D), F32) for n in ("x", "dx")}
    src["lse"] = torch.full((t.H, t.Lp), 9.0, device=DEV)
    buf = {n: torch.zeros_like(a) for n, a in src.items()}
    ws = {op: t.ws(op) for op in range(5)}
    e = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731

    def outputs(make):
        def of(fn):
            fn.outputs = make
            return fn
        return of

    @outputs(lambda: (e(t.Lp, t.D, dt=F32), e(3, 6, t.D)))
    def adaln(b, stream, out):
        h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, b["x"], mod, 0, b["xm"], b["dx"], *out, ws[0], stream)

    @outputs(lambda: (e(t.Lp, t.D), e(3 * t.I, t.D), e(128), e(128)))
    def qkv(b, stream, out):
        h3.h3_qkv_qknorm_mrope_backward(t.dims, t.ranges, b["xm"], W["qkv"], w, w, pos, b["q"], b["k"], b["v"], *out,
                                        ws[1], stream)

    @outputs(lambda: tuple(e(t.H, t.Lp, 128) for _ in range(3)))
    def attention(b, stream, out):
        h3.h3_attention_backward(t.dims, t.ranges, b["q"], b["k"], b["v"], b["o"], b["lse"], b["do"], *out, ws[2],
                                 stream)

    @outputs(lambda: (e(t.Lp, t.I), e(t.D, t.I), e(3, 6, t.D)))
    def gated(b, stream, out):
        h3.h3_gated_residual_backward(t.dims, t.ranges, b["dx"], b["o"], W["o"], mod, *out, ws[3], stream=stream)

    @outputs(lambda: (e(t.Lp, t.D), e(2 * t.F, t.D), e(t.D, t.F), e(3, 6, t.D)))
    def ffn(b, stream, out):
        h3.h3_ffn_swiglu_backward(t.dims, t.ranges, b["dx"], b["xm"], W["gu"], W["d"], mod, *out, ws[4], stream)

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    for call in (adaln, qkv, attention, gated, ffn):
        want = call.outputs()
        call(src, None, want)
        torch.cuda.synchronize()
        for kind in ("copy", "memset", "join"):
            for b in buf.values():
                b.zero_()
            torch.cuda.synchronize()
            got, graph = call.outputs(), torch.cuda.CUDAGraph()  # outputs first: the call follows the copies
            with torch.cuda.graph(graph, stream=main):
                if kind == "join":
                    side.wait_stream(main)
                    with torch.cuda.stream(side):
                        for n in buf:
                            buf[n].copy_(src[n])
                    main.wait_stream(side)
                    call(buf, main, got)
                else:
                    for n in buf:
                        if kind == "memset":
                            buf[n].zero_()
                        else:
                            buf[n].copy_(src[n])
                    call(buf, main, got)
            for _ in range(2):
                for b in buf.values():
                    b.fill_(3.0)
                for g in got:
                    g.fill_(1.0)
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                same = want
                if kind == "memset":
                    same = call.outputs()
                    call(buf, None, same)
                    torch.cuda.synchronize()
                for g, r in zip(got, same):
                    if g.shape == (3, 6, t.D):  # slots that are not the call's hold what stood there
                        mine = (r != 0).any(-1)
                        g, r = g[mine], r[mine]
                    assert torch.equal(g, r), (call.__name__, kind)
    t.finish()


# ---------------------------------------------------------------- refusals

def test_python_forms_check_sizes_types_and_workspace():
    t = Inputs((10, 0, 20), 64, 1, 128, fill=0.0)
    f, b = torch.zeros(t.Lp, 64, device=DEV), torch.zeros(t.Lp, 64, dtype=BF16, device=DEV)
    mod, ws = torch.zeros(3, 6, 64, device=DEV), t.ws(h3.H3_BWD_ADALN)
    call = lambda **kw: h3.h3_adaln_norm_modulate_backward(  # noqa: E731
        t.dims, t.ranges, kw.get("x", f), mod, 0, kw.get("dxm", b), f, kw.get("dx", torch.zeros_like(f)),
        kw.get("dmod"), kw.get("ws", ws))
    call()
    for kw, exc in (({"x": f[:1]}, ValueError), ({"x": b}, TypeError), ({"dxm": b.T.contiguous().T}, ValueError),
                    ({"dmod": torch.zeros(18, dtype=BF16, device=DEV)}, ValueError), ({"ws": ws[:16]}, ValueError),
                    ({"dx": f.cpu()}, TypeError), ({"x": None}, TypeError), ({"ws": None}, TypeError),
                    ({"dx": f[:, :]}, None)):
        if exc is None:
            continue
        with pytest.raises(exc):
            call(**kw)
    with pytest.raises(h3.H3Error):
        h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, f, mod, 2, b, f, torch.zeros_like(f), None, ws)
    with pytest.raises(h3.H3Error):  # dx over x
        h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, f, mod, 0, b, torch.zeros_like(f), f, None, ws)
    t.finish()
