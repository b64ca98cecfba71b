"""Float64 CPU oracle of the block's backward pass.  TEST INFRASTRUCTURE ONLY.

The gradients of oracle.h3_oracle's forward functions, written as formulas in
NumPy float64 and pinned to central differences of those functions by
tests/test_oracle_bwd_pins.py.  Arrays hold the L valid tokens; modalities
without tokens get gradients of 0.  No code is shared with the CUDA library.

With `err=True` a function also returns, element by element, a bound on what an
implementation may be off that keeps its sums in fp32 and rounds to bf16 (half a
step: U = 2^-8 relative) the operands of its matrix products that the inputs do
not already give in bf16, and its bf16 results once.  The bounds carry every
such rounding through sums of absolute values, so they hold whatever the signs;
ACC covers fp32 accumulation and exponentials.
"""
from __future__ import annotations

import numpy as np

from .h3_oracle import (EPS_LN, EPS_QK, GATE, MLP, MSA, SCALE, modality_of_rows, rope_angles)

U = 2.0 ** -8
ACC = 2.0 ** -14  # relative to a sum of absolute values; fp32 sums of up to 10^5 terms stay far below it


def _f(a):
    return np.asarray(a, np.float64)


def _by_modality(ranges, t):
    """Sums of rows over each modality, [3][D]."""
    m = modality_of_rows(ranges)
    return np.stack([t[m == i].sum(axis=0) for i in range(3)])


def adaln_modulate(x, mod, ranges, branch, dy, dres, err=False):
    """(dx, dshift, dscale) of h3_oracle.adaln_modulate, dx joined with the
    residual's gradient dres."""
    x, mod, dy, dres = _f(x), _f(mod), _f(dy), _f(dres)
    mu = x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mu) ** 2).mean(axis=1, keepdims=True) + EPS_LN)
    xhat = (x - mu) * rstd
    dh = dy * (1.0 + mod[modality_of_rows(ranges), 3 * branch + SCALE])
    dx = dres + rstd * (dh - dh.mean(axis=1, keepdims=True) - xhat * (dh * xhat).mean(axis=1, keepdims=True))
    dshift, dscale = _by_modality(ranges, dy), _by_modality(ranges, dy * xhat)
    if not err:
        return dx, dshift, dscale
    a = np.abs(dh)
    # x - mu loses what x rounds off at fp32 against the row's spread
    spread = 2.0 ** -22 * (np.abs(x).max(axis=1, keepdims=True) * rstd + 1.0)
    e_dx = 2.0 ** -22 * np.abs(dres) + (2.0 ** -20 + spread) * rstd * (
        a + a.mean(axis=1, keepdims=True) + (np.abs(xhat) + 1.0) * (a * (np.abs(xhat) + 1.0)).mean(axis=1, keepdims=True))
    return ((dx, e_dx), (dshift, U * np.abs(dshift) + ACC * _by_modality(ranges, np.abs(dy))),
            (dscale, U * np.abs(dscale) + _by_modality(ranges, (ACC + spread) * np.abs(dy) * (np.abs(xhat) + 1.0))))


def unrotate(d, pos, split=(32, 48, 48)):
    """The transpose of h3_oracle.rope: every pair turned back."""
    ang = rope_angles(_f(pos), split)[:, None, :]
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty_like(d)
    out[..., 0::2] = d[..., 0::2] * c + d[..., 1::2] * s
    out[..., 1::2] = d[..., 1::2] * c - d[..., 0::2] * s
    return out


def qkv_qknorm_mrope(xm, Wqkv, qn_w, kn_w, pos, n_heads, dq, dk, dv, split=(32, 48, 48), err=False):
    """(dxm, dWqkv, dqn_w, dkn_w) of h3_oracle.qkv_qknorm_mrope; dq, dk, dv
    [L, heads, 128]."""
    xm, W = _f(xm), _f(Wqkv)
    L, I = xm.shape[0], n_heads * 128
    raw = (xm @ W.T).reshape(L, 3, n_heads, 128)
    raw_abs = (np.abs(xm) @ np.abs(W).T).reshape(L, 3, n_heads, 128)
    parts, errs, dws = [], [], []
    for i, (d, w) in enumerate(((dq, qn_w), (dk, kn_w))):
        t, w, x = unrotate(_f(d), pos, split), _f(w), raw[:, i]
        rstd = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + EPS_QK)
        xhat = x * rstd
        dh = t * w
        m = (dh * xhat).mean(axis=-1, keepdims=True)
        parts.append(rstd * (dh - xhat * m))
        dw = (t * xhat).sum(axis=(0, 1))
        if err:
            # fp32 angles move t by up to 2^-16 of its pair; raw carries its own sums' error
            ta = np.repeat(np.hypot(t[..., 0::2], t[..., 1::2]), 2, axis=-1)
            rel = ACC * (1.0 + raw_abs[:, i] * rstd)
            ha = ta * np.abs(w)
            ma = (ha * (np.abs(xhat) + 1.0)).mean(axis=-1, keepdims=True)
            errs.append(U * np.abs(parts[-1]) + rel * rstd * (ha + (np.abs(xhat) + 1.0) * ma))
            dws.append((dw, U * np.abs(dw) + (rel * ta * (np.abs(xhat) + 1.0)).sum(axis=(0, 1))))
        else:
            dws.append(dw)
    parts.append(_f(dv))
    dqkv = np.stack(parts, axis=1).reshape(L, 3 * I)
    dxm, dW = dqkv @ W, dqkv.T @ xm
    if not err:
        return dxm, dW, dws[0], dws[1]
    e = np.stack(errs + [np.zeros_like(errs[0])], axis=1).reshape(L, 3 * I) + ACC * np.abs(dqkv)
    return ((dxm, U * np.abs(dxm) + e @ np.abs(W)), (dW, U * np.abs(dW) + e.T @ np.abs(xm)), dws[0], dws[1])


def attention_lse(q, k):
    """log sum_j exp(q_i k_j / sqrt(128)) per head, [heads, L]; q, k [L, heads, 128]."""
    s = np.einsum("ihd,jhd->hij", _f(q), _f(k)) / np.sqrt(128.0)
    top = s.max(axis=2, keepdims=True)
    return (top + np.log(np.exp(s - top).sum(axis=2, keepdims=True)))[..., 0]


def attention(q, k, v, do, err=False):
    """(dq, dk, dv) of h3_oracle.attention; all [L, heads, 128]."""
    q, k, v, do = (_f(a).transpose(1, 0, 2) for a in (q, k, v, do))
    c = 1.0 / np.sqrt(128.0)
    s = c * (q @ k.transpose(0, 2, 1))
    top = s.max(axis=2, keepdims=True)
    p = np.exp(s - top)
    p /= p.sum(axis=2, keepdims=True)
    o = p @ v
    dv = p.transpose(0, 2, 1) @ do
    dp = do @ v.transpose(0, 2, 1)
    ds = p * (dp - (do * o).sum(axis=2, keepdims=True))
    dq, dk = c * (ds @ k), c * (ds.transpose(0, 2, 1) @ q)
    back = lambda *ts: tuple(t.transpose(1, 0, 2) for t in ts)  # noqa: E731
    if not err:
        return back(dq, dk, dv)
    qa, ka, va, da = (np.abs(t) for t in (q, k, v, do))
    # p: fp32 scores and exponentials; ds: P and o rounded to bf16, ds rounded once
    ep = p * (2.0 ** -20 * (1.0 + np.abs(s) + c * (qa @ ka.transpose(0, 2, 1))))
    # o itself carries its forward pass: P rounded to bf16 and o rounded once
    e_o = U * np.abs(o) + (U * p + ep) @ va
    e_delta = (da * (e_o + ACC * np.abs(o))).sum(axis=2, keepdims=True)
    dpa = da @ va.transpose(0, 2, 1)
    e_ds = U * np.abs(ds) + p * (e_delta + ACC * dpa) + ep * (dpa + (da * np.abs(o)).sum(axis=2, keepdims=True))
    e_dv = U * np.abs(dv) + (U * p + ACC * p + ep).transpose(0, 2, 1) @ da
    e_dq = U * np.abs(dq) + c * ((e_ds + ACC * np.abs(ds)) @ ka)
    e_dk = U * np.abs(dk) + c * ((e_ds + ACC * np.abs(ds)).transpose(0, 2, 1) @ qa)
    return tuple(zip(back(dq, dk, dv), back(e_dq, e_dk, e_dv)))


def _gated(dx, b, W, mod, ranges, branch, e_b, err):
    """(db, dW, dgate) of gate_m (.) (b W^T); e_b: how far b may be off."""
    dx, b, W = _f(dx), _f(b), _f(W)
    gate = _f(mod)[modality_of_rows(ranges), 3 * branch + GATE]
    dy = gate * dx
    db, dW, dgate = dy @ W, dy.T @ b, _by_modality(ranges, dx * (b @ W.T))
    if not err:
        return db, dW, dgate
    ya, ba, Wa, xa = np.abs(dy), np.abs(b), np.abs(W), np.abs(dx)
    e_db = (U + ACC) * (ya @ Wa)
    e_dW = U * np.abs(dW) + (U + ACC) * (ya.T @ ba) + ya.T @ e_b
    e_gate = U * np.abs(dgate) + _by_modality(ranges, xa * (((U + ACC) * ba + e_b) @ Wa.T))
    return (db, e_db), (dW, e_dW), (dgate, e_gate)


def gated_residual(dx, o, Wo, mod, ranges, branch=MSA, err=False):
    """(do, dWo, dgate) of h3_oracle.gated_residual."""
    out = _gated(dx, o, Wo, mod, ranges, branch, np.zeros_like(_f(o)), err)
    if err:
        (do, e), dW, dg = out
        return (do, e + U * np.abs(do)), dW, dg
    return out


def ffn_swiglu(dx, xm, Wgu, Wd, mod, ranges, err=False):
    """(dxm, dWgu, dWd, dgate) of h3_oracle.ffn_swiglu."""
    xm, Wgu = _f(xm), _f(Wgu)
    F = Wgu.shape[0] // 2
    gu = xm @ Wgu.T
    g, u = gu[:, :F], gu[:, F:]
    sig = 1.0 / (1.0 + np.exp(-g))
    act, dact = g * sig, sig * (1.0 + g * (1.0 - sig))
    h = act * u
    if not err:
        dh, dWd, dgate = _gated(dx, h, Wd, mod, ranges, MLP, None, False)
        dgu = np.concatenate([dh * u * dact, dh * act], axis=1)
        return dgu @ Wgu, dgu.T @ xm, dWd, dgate
    e_gu = ACC * (np.abs(xm) @ np.abs(Wgu).T)
    e_g, e_u = e_gu[:, :F], e_gu[:, F:]
    # |act'| <= 1.1, |act''| <= 0.5
    e_h = U * np.abs(h) + 1.1 * e_g * np.abs(u) + np.abs(act) * e_u + ACC * np.abs(h)
    (dh, e_dh), dWd, dgate = _gated(dx, h, Wd, mod, ranges, MLP, e_h, True)
    dg, du = dh * u * dact, dh * act
    e_dg = (U + ACC) * np.abs(dg) + e_dh * np.abs(u * dact) + np.abs(dh) * (e_u * np.abs(dact) + 0.5 * np.abs(u) * e_g)
    e_du = (U + ACC) * np.abs(du) + e_dh * np.abs(act) + 1.1 * np.abs(dh) * e_g
    dgu, e = np.concatenate([dg, du], axis=1), np.concatenate([e_dg, e_du], axis=1)
    e = e + ACC * np.abs(dgu)
    dxm, dWgu = dgu @ Wgu, dgu.T @ xm
    return ((dxm, U * np.abs(dxm) + e @ np.abs(Wgu)), (dWgu, U * np.abs(dWgu) + e.T @ np.abs(xm)), dWd, dgate)


def block(x, mod, ranges, pos, Wqkv, qn_w, kn_w, Wo, Wgu, Wd, n_heads, dx):
    """Gradients of h3_oracle.block_forward: (dx, {weight or "mod": gradient})."""
    from . import h3_oracle as O
    _, p = O.block_forward(x, mod, ranges, pos, Wqkv, qn_w, kn_w, Wo, Wgu, Wd, n_heads, return_parts=True)
    L = p["q"].shape[0]
    dmod = np.zeros((3, 6) + _f(x).shape[1:])
    g = {"mod": dmod}
    dxm, g["Wgu"], g["Wd"], dmod[:, 5] = ffn_swiglu(dx, p["xm2"], Wgu, Wd, mod, ranges)
    dx, dmod[:, 3], dmod[:, 4] = adaln_modulate(p["x1"], mod, ranges, MLP, dxm, dx)
    do, g["Wo"], dmod[:, 2] = gated_residual(dx, p["o"], Wo, mod, ranges)
    dq, dk, dv = attention(p["q"], p["k"], p["v"], do.reshape(L, n_heads, 128))
    dxm, g["Wqkv"], g["qn_w"], g["kn_w"] = qkv_qknorm_mrope(p["xm1"], Wqkv, qn_w, kn_w, pos, n_heads, dq, dk, dv)
    dx, dmod[:, 0], dmod[:, 1] = adaln_modulate(x, mod, ranges, MSA, dxm, dx)
    return dx, g
