"""The backward oracle's formulas against central differences of the forward
oracle: for a random direction, the derivative of sum(gradient . output) along
it, and for the whole block the same through every weight."""
import numpy as np
import pytest

from oracle import h3_oracle as O
from oracle import h3_oracle_bwd as G

RANGES = [O.pack_ranges(3, 2, 6), O.pack_ranges(0, 0, 1), O.pack_ranges(5, 0, 4)]
D, H, F = 64, 2, 128
STEP = 1e-5


def differences(f, args, which, directions):
    """d/dt f(args + t directions) at 0 for the arguments in `which`."""
    at = lambda t: f(*[a + t * directions[i] if i in which else a for i, a in enumerate(args)])  # noqa: E731
    return (at(STEP) - at(-STEP)) / (2 * STEP)


def check(f, args, grads, rng):
    """grads: {argument index: gradient of sum(f)}."""
    dirs = {i: rng.standard_normal(args[i].shape) for i in grads}
    for i, g in grads.items():
        num = differences(f, args, {i}, dirs)
        ana = float((g * dirs[i]).sum())
        # O(h^2) truncation and 1e-16 / h rounding of values of order 1 to 100
        assert abs(num - ana) <= 1e-6 * (1.0 + abs(ana)), (i, num, ana)


@pytest.mark.parametrize("r", RANGES, ids=lambda r: str(r["count"]))
@pytest.mark.parametrize("branch", (O.MSA, O.MLP))
def test_adaln(r, branch):
    rng = np.random.default_rng(1)
    L = r["L"]
    x, mod, dy = rng.standard_normal((L, D)), 0.3 * rng.standard_normal((3, 6, D)), rng.standard_normal((L, D))
    dx, dshift, dscale = G.adaln_modulate(x, mod, r, branch, dy, np.zeros((L, D)))
    dmod = np.zeros_like(mod)
    dmod[:, 3 * branch], dmod[:, 3 * branch + 1] = dshift, dscale
    check(lambda x, mod: float((O.adaln_modulate(x, mod, r, branch) * dy).sum()), [x, mod], {0: dx, 1: dmod}, rng)
    res = rng.standard_normal((L, D))
    assert np.allclose(G.adaln_modulate(x, mod, r, branch, dy, res)[0], dx + res)


def test_qkv():
    rng = np.random.default_rng(2)
    r = RANGES[0]
    L = r["L"]
    pos = rng.uniform(0, 20, (L, 3))
    xm, W = rng.standard_normal((L, D)), 0.2 * rng.standard_normal((3 * H * 128, D))
    qn, kn = 1 + 0.1 * rng.standard_normal(128), 1 + 0.1 * rng.standard_normal(128)
    ds = [rng.standard_normal((L, H, 128)) for _ in range(3)]
    grads = G.qkv_qknorm_mrope(xm, W, qn, kn, pos, H, *ds)
    f = lambda xm, W, qn, kn: float(sum((a * b).sum() for a, b in  # noqa: E731
                                        zip(O.qkv_qknorm_mrope(xm, W, qn, kn, pos, H), ds)))
    check(f, [xm, W, qn, kn], dict(enumerate(grads)), rng)


@pytest.mark.parametrize("L", (1, 2, 9))
def test_attention(L):
    rng = np.random.default_rng(3)
    q, k, v, do = (rng.standard_normal((L, H, 128)) for _ in range(4))
    f = lambda q, k, v: float((O.attention(q, k, v) * do.reshape(L, -1)).sum())  # noqa: E731
    check(f, [q, k, v], dict(enumerate(G.attention(q, k, v, do))), rng)
    s = np.einsum("ihd,jhd->hij", q, k) / np.sqrt(128)
    assert np.allclose(np.exp(s - G.attention_lse(q, k)[..., None]).sum(axis=2), 1.0)


@pytest.mark.parametrize("r", RANGES, ids=lambda r: str(r["count"]))
def test_gated_branches(r):
    rng = np.random.default_rng(4)
    L = r["L"]
    x, dx, mod = rng.standard_normal((L, D)), rng.standard_normal((L, D)), rng.standard_normal((3, 6, D))
    o, Wo = rng.standard_normal((L, H * 128)), 0.1 * rng.standard_normal((D, H * 128))
    do, dWo, dg = G.gated_residual(dx, o, Wo, mod, r)
    dmod = np.zeros_like(mod)
    dmod[:, 2] = dg
    f = lambda o, Wo, mod: float((O.gated_residual(x, o, Wo, mod, r) * dx).sum())  # noqa: E731
    check(f, [o, Wo, mod], {0: do, 1: dWo, 2: dmod}, rng)
    xm, Wgu, Wd = rng.standard_normal((L, D)), 0.2 * rng.standard_normal((2 * F, D)), 0.1 * rng.standard_normal((D, F))
    dxm, dWgu, dWd, dg = G.ffn_swiglu(dx, xm, Wgu, Wd, mod, r)
    dmod = np.zeros_like(mod)
    dmod[:, 5] = dg
    f = lambda xm, Wgu, Wd, mod: float((O.ffn_swiglu(x, xm, Wgu, Wd, mod, r) * dx).sum())  # noqa: E731
    check(f, [xm, Wgu, Wd, mod], {0: dxm, 1: dWgu, 2: dWd, 3: dmod}, rng)


def test_block():
    rng = np.random.default_rng(5)
    r = RANGES[0]
    L = r["L"]
    pos = rng.uniform(0, 5, (L, 3))
    x, mod, dx = rng.standard_normal((L, D)), 0.3 * rng.standard_normal((3, 6, D)), rng.standard_normal((L, D))
    W = {"Wqkv": 0.2 * rng.standard_normal((3 * H * 128, D)), "qn_w": 1 + 0.1 * rng.standard_normal(128),
         "kn_w": 1 + 0.1 * rng.standard_normal(128), "Wo": 0.1 * rng.standard_normal((D, H * 128)),
         "Wgu": 0.2 * rng.standard_normal((2 * F, D)), "Wd": 0.1 * rng.standard_normal((D, F))}
    names = list(W)
    dx0, g = G.block(x, mod, r, pos, *W.values(), H, dx)
    f = lambda x, mod, *ws: float((O.block_forward(x, mod, r, pos, *ws, H) * dx).sum())  # noqa: E731
    grads = {0: dx0, 1: g["mod"], **{2 + i: g[n] for i, n in enumerate(names)}}
    check(f, [x, mod, *W.values()], grads, rng)


def test_error_bounds_hold_for_rounded_operands():
    """The bounds of err=True against a float64 emulation that rounds what an
    implementation rounds (the feed-forward: gated gradient, h, dgate/dup, and
    the results), so that they are neither vacuous nor too tight."""
    rng = np.random.default_rng(6)
    r = O.pack_ranges(20, 13, 67)
    L = r["L"]
    b16 = lambda a: O.round_to_bf16(np.asarray(a, np.float32)).astype(np.float64)  # noqa: E731
    dx, mod = rng.standard_normal((L, D)), rng.standard_normal((3, 6, D))
    xm, Wgu, Wd = (b16(a) for a in (rng.standard_normal((L, D)), 0.2 * rng.standard_normal((2 * F, D)),
                                    0.1 * rng.standard_normal((D, F))))
    gate = mod[O.modality_of_rows(r), 5]
    gu = xm @ Wgu.T
    g, u = gu[:, :F], gu[:, F:]
    sig = 1 / (1 + np.exp(-g))
    h = b16(g * sig * u)
    dh = b16(gate * dx) @ Wd
    dgu = b16(np.concatenate([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1))
    m = O.modality_of_rows(r)
    per = np.stack([b16(dx)[m == i].T @ h[m == i] for i in range(3)])
    got = [b16(dgu @ Wgu), b16(dgu.T @ xm), b16((mod[:, 5][..., None] * per).sum(0)), b16((per * Wd).sum(2))]
    for a, (ref, e) in zip(got, G.ffn_swiglu(dx, xm, Wgu, Wd, mod, r, err=True)):
        assert np.all(np.abs(a - ref) <= e)
        assert np.abs(a - ref).max() >= 0.02 * e.max()
