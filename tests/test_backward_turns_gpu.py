"""Backward calls where a CTA, or a pair of them, takes many turns: several
tiles of the QKV kernel, separate launches of full-width products, the AdaLN
ring of stages; and the packing's modalities in another order.

Tolerances as in test_backward_gpu: the oracle's element-wise bounds, and the
2-norm within one half step of bf16 (U) for each rounding on the way."""
import numpy as np
import pytest
import torch

from oracle import h3_oracle_bwd as G
from omni_modal_diffusion_b200 import h3

from test_backward_gpu import BF16, DEV, F32, U, Inputs, check_adaln, dev, inside, mod_with_zero_gates

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from omni_modal_diffusion_b200 import build
    build.build()
    assert torch.cuda.is_available()


def qkv_call(t, xm, W, qn, kn, pos, ds):
    out = [t.empty(t.Lp, t.D), t.empty(3 * t.I, t.D), t.empty(128), t.empty(128)]
    h3.h3_qkv_qknorm_mrope_backward(t.dims, t.ranges, xm, W, qn, kn, pos, *ds, *out, t.ws(h3.H3_BWD_QKV))
    t.finish()
    return out


def check_qkv(t, seed_pos=90):
    xm, W = t.normal(t.L, t.D), t.normal(3 * t.I, t.D, std=0.05)
    qn, kn = t.normal(128, std=0.1, mean=1.0), t.normal(128, std=0.1, mean=1.0)
    pos = t.rng.integers(0, seed_pos, (t.L, 3)).astype(np.float32)
    ds = [t.normal(t.L, t.H, 128, std=s) for s in (1e-3, 1e-2, 1.0)]
    out = qkv_call(t, t.rows(xm), dev(W), dev(qn), dev(kn), t.rows(pos, F32), [t.heads(d) for d in ds])
    want = G.qkv_qknorm_mrope(xm, W, qn, kn, pos, t.H, *ds, err=True)
    inside(out[0][:t.L], want[0], "dxm", 2)
    assert torch.all(out[0][t.L:] == 0)
    for got, w, name, n in zip(out[1:], want[1:], ("dWqkv", "dqn_w", "dkn_w"), (2, 1.1, 1.1)):
        inside(got, w, name, n)


@pytest.mark.parametrize("counts,D,H", (((300, 0, 2300), 128, 16), ((0, 77, 1500), 64, 45)), ids=str)
def test_qkv_several_tiles_for_each_pair(counts, D, H):
    """11 x 16 and 7 x 45 tiles of the norm's kernel for 74 CTA pairs: both TMEM
    accumulators and both halves of the exchange buffer in turn, the norm
    weights' sums over a pair's tiles."""
    check_qkv(Inputs(counts, D, H, 128, seed=H))


# ---------------------------------------------------------------- full width, a launch for each product

def rows_and_columns(got, ref, roundings, name):
    """Every row's and every column's error within its own norm's share: one
    tile, row or column in the wrong place does not hide behind the others."""
    off = (got.double() - ref).square_()
    ref = ref.square()
    for dim in (0, 1):
        lim = (roundings * U) ** 2 * ref.sum(dim)
        assert torch.all(off.sum(dim) <= lim), (name, dim, float((off.sum(dim) / ref.sum(dim)).max().sqrt()))


WIDE = (300, 131, 2469)  # 2,900 tokens: 165 K and 380 K k blocks, above what shares a launch


def wide(seed):
    t = Inputs(WIDE, 5376, 56, 14336, seed=seed, fill=0.0)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0, dt=BF16, rows=None):
        a = torch.empty(*s, device=DEV, dtype=F32).normal_(mean, std, generator=g).to(dt)
        if rows is not None:
            a.narrow(rows, t.L, t.Lp - t.L).fill_(float("nan"))  # padding rows are not read
        return a

    return t, normal


def test_qkv_full_width():
    t, normal = wide(141)
    L, D, H, I = t.L, t.D, t.H, t.I
    xm, W, qn, kn = normal(t.Lp, D, rows=0), normal(3 * I, D, std=0.02), normal(128, std=0.1, mean=1), normal(128, std=0.1, mean=1)
    pos = torch.zeros(t.Lp, 3, device=DEV)
    pos[:L] = dev(t.rng.integers(0, 40, (L, 3)), F32)
    ds = [normal(H, t.Lp, 128, std=1e-3, rows=1) for _ in range(3)]
    dxm, dW, dqn, dkn = qkv_call(t, xm, W, qn, kn, pos, ds)
    x, Wd = xm[:L].double(), W.double()
    freq = torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) for d in (32, 48, 48)]).to(DEV)
    axis = torch.tensor([0] * 16 + [1] * 24 + [2] * 24, device=DEV)
    ang = (pos[:L].double()[:, axis] * freq)[:, None]
    c, s = ang.cos(), ang.sin()
    dqkv = torch.empty(L, 3, H, 128, device=DEV, dtype=torch.float64)
    for i, (d, w, dw) in enumerate(((ds[0], qn, dqn), (ds[1], kn, dkn))):
        d = d[:, :L].double().transpose(0, 1)
        a, b = d[..., 0::2], d[..., 1::2]
        turned = torch.stack((a * c + b * s, b * c - a * s), -1).flatten(-2)
        raw = (x @ Wd[i * I:(i + 1) * I].T).view(L, H, 128)
        inv = torch.rsqrt(raw.square().mean(-1, keepdim=True) + 1e-6)
        xhat, dh = raw * inv, turned * w.double()
        ref = (turned * xhat).sum((0, 1))
        assert (dw.double() - ref).norm() <= 1.1 * U * ref.norm()
        dqkv[:, i] = inv * (dh - xhat * (dh * xhat).mean(-1, keepdim=True))
    dqkv[:, 2] = ds[2][:, :L].double().transpose(0, 1)
    dqkv = dqkv.view(L, 3 * I)
    rows_and_columns(dxm[:L], dqkv @ Wd, 2, "dxm")
    assert torch.all(dxm[L:] == 0)
    rows_and_columns(dW, dqkv.T @ x, 2, "dWqkv")


def test_ffn_full_width():
    t, normal = wide(151)
    L, D, F = t.L, t.D, t.F
    dx, xm, mod = normal(t.Lp, D, dt=F32, rows=0), normal(t.Lp, D, rows=0), normal(3, 6, D, std=0.3, dt=F32)
    Wgu, Wd = normal(2 * F, D, std=0.02), normal(D, F, std=0.02)
    dxm, dWgu, dWd, dmod = t.empty(t.Lp, D), t.empty(2 * F, D), t.empty(D, F), t.empty(3, 6, D)
    h3.h3_ffn_swiglu_backward(t.dims, t.ranges, dx, xm, Wgu, Wd, mod, dxm, dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
    t.finish()
    x, d = xm[:L].double(), dx[:L].double()
    g, u = x @ Wgu[:F].double().T, x @ Wgu[F:].double().T
    sig = torch.sigmoid(g)
    h = g * sig * u
    dy = d * torch.repeat_interleave(mod[:, 5].double(), torch.tensor(WIDE, device=DEV), dim=0)
    dh = dy @ Wd.double()
    dgu = torch.cat((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), 1)
    rows_and_columns(dxm[:L], dgu @ Wgu.double(), 3, "dxm")
    assert torch.all(dxm[L:] == 0)
    rows_and_columns(dWgu, dgu.T @ x, 3, "dWgu")
    rows_and_columns(dWd, dy.T @ h, 3, "dWd")
    y = d * (h @ Wd.double().T)
    gate = torch.stack([p.sum(0) for p in y.split(WIDE)])
    for m in range(3):
        assert (dmod[m, 5].double() - gate[m]).norm() <= 3 * U * gate[m].norm(), m
    assert torch.all(torch.isnan(dmod[:, :5].float()))


# ---------------------------------------------------------------- AdaLN

@pytest.mark.parametrize("D,counts", ((1024, (1500, 3, 5010)), (2112, (7, 2000, 4001)), (5376, (513, 1, 2790)),
                                      (8192, (1, 700, 803))), ids=str)
def test_adaln_many_rows_in_a_ring_of_few_stages(D, counts):
    """One to four columns a thread, several warps a CTA and some ten rows for
    each, through four, three, two and two stages; the modalities' last CTAs
    are short."""
    t = Inputs(counts, D, 1, 128, seed=D)
    check_adaln(t, 1, t.normal(t.L, D, std=3.0, mean=0.5, bf16=False), t.normal(3, 6, D, std=0.1, bf16=False),
                t.normal(t.L, D, std=1e-3), t.normal(t.L, D, std=1e-3, bf16=False), in_place=D == 5376)


# ---------------------------------------------------------------- modalities in another order

ORDERS = ((2, 1, 0), (1, 2, 0), (2, 0, 1))


def reorder(t, order):
    """The packing with its modalities one after another in `order`."""
    at = 0
    for m in order:
        t.ranges.start[m] = t.r["start"][m] = at
        at += t.r["count"][m]


@pytest.mark.parametrize("order", ORDERS, ids=str)
@pytest.mark.parametrize("counts", ((37, 58, 240), (5, 0, 252), (300, 130, 70)), ids=str)
def test_modalities_in_another_order(counts, order):
    D, H, F = 320, 2, 384
    t = Inputs(counts, D, H, F, seed=sum(counts))
    reorder(t, order)
    check_adaln(t, 0, t.normal(t.L, D, std=3.0, bf16=False), t.normal(3, 6, D, std=0.1, bf16=False), t.normal(t.L, D),
                t.normal(t.L, D, bf16=False))
    dx, o, Wo, mod = t.normal(t.L, D, bf16=False), t.normal(t.L, t.I), t.normal(D, t.I, std=0.05), mod_with_zero_gates(t)
    do, dWo, dmod = t.empty(t.Lp, t.I), t.empty(D, t.I), t.empty(3, 6, D)
    h3.h3_gated_residual_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(o), dev(Wo), dev(mod, F32), do, dWo, dmod,
                                  t.ws(h3.H3_BWD_GATED_RESIDUAL))
    t.finish()
    want = G.gated_residual(dx, o, Wo, mod, t.r, err=True)
    for got, w, name in zip((do[:t.L], dWo, dmod[:, 2]), want, ("do", "dWo", "dgate")):
        inside(got, w, name, 2)
    xm, Wgu, Wd = t.normal(t.L, D), t.normal(2 * F, D, std=0.1), t.normal(D, F, std=0.05)
    dxm, dWgu, dWd, dmod = t.empty(t.Lp, D), t.empty(2 * F, D), t.empty(D, F), t.empty(3, 6, D)
    h3.h3_ffn_swiglu_backward(t.dims, t.ranges, t.rows(dx, F32), t.rows(xm), dev(Wgu), dev(Wd), dev(mod, F32), dxm,
                              dWgu, dWd, dmod, t.ws(h3.H3_BWD_FFN))
    t.finish()
    want = G.ffn_swiglu(dx, xm, Wgu, Wd, mod, t.r, err=True)
    for got, w, name in zip((dxm[:t.L], dWgu, dWd, dmod[:, 5]), want, ("dxm", "dWgu", "dWd", "dgate")):
        inside(got, w, name, 3)


# ---------------------------------------------------------------- a call's own slots, views

def test_captured_calls_write_their_own_modulation_slots():
    """Captured behind memsets that leave every input 0: the replay writes 0
    into the call's own slots of dmod, for every modality, and no others."""
    D, H, F = 320, 2, 384
    t = Inputs((37, 0, 90), D, H, F, seed=161, fill=0.0)
    e = lambda *s, dt=BF16: torch.ones(*s, dtype=dt, device=DEV)  # noqa: E731
    f, b, o = e(t.Lp, D, dt=F32), e(t.Lp, D), e(t.Lp, t.I)
    mod, Wo, Wgu, Wd = e(3, 6, D, dt=F32), e(D, t.I), e(2 * F, D), e(D, F)
    ws = t.ws(h3.H3_BWD_FFN), t.ws(h3.H3_BWD_GATED_RESIDUAL), t.ws(h3.H3_BWD_ADALN)
    out_f, out_b, out_o = e(t.Lp, D, dt=F32), e(t.Lp, D), e(t.Lp, t.I)
    dmod = e(3, 6, D)
    calls = {
        (0, 1): lambda: h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, f, mod, 0, b, f, out_f, dmod, ws[2]),
        (3, 4): lambda: h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, f, mod, 1, b, f, out_f, dmod, ws[2]),
        (2,): lambda: h3.h3_gated_residual_backward(t.dims, t.ranges, f, o, Wo, mod, out_o, None, dmod, ws[1]),
        (5,): lambda: h3.h3_ffn_swiglu_backward(t.dims, t.ranges, f, b, Wgu, Wd, mod, out_b, None, None, dmod, ws[0]),
    }
    for slots, call in calls.items():
        call()  # function attributes are set before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for a in (f, b, o):
                a.zero_()
            call()
        for _ in range(2):
            for a in (f, b, o, dmod):
                a.fill_(1.0)
            graph.replay()
            torch.cuda.synchronize()
            for i in range(6):
                assert torch.all(dmod[:, i] == (0.0 if i in slots else 1.0)), (slots, i)
    t.finish()


def test_contiguous_views_are_accepted():
    t = Inputs((10, 0, 20), 64, 1, 128, fill=0.0)
    x, dy, res = t.normal(t.L, 64, bf16=False), t.normal(t.L, 64), t.normal(t.L, 64, bf16=False)
    mod = dev(t.normal(3, 6, 64, bf16=False), F32)
    gx, gdy, gres = t.rows(x, F32), t.rows(dy), t.rows(res, F32)
    want, dx, big = torch.empty_like(gx), torch.empty(3, t.Lp, 64, device=DEV), torch.stack((gres, gx, gres))
    ws = t.ws(h3.H3_BWD_ADALN)
    h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, gx, mod, 0, gdy, gres, want, None, ws)
    h3.h3_adaln_norm_modulate_backward(t.dims, t.ranges, big[1][:, :], mod.view(18, 64), 0, gdy.view(-1), big[2], dx[1], None,
                                       ws)
    t.finish()
    assert torch.equal(dx[1], want)
