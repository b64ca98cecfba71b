"""Cases and plain forms of the block's backward pass.

The operators are the gradients of the block's five calls: the AdaLN norm and
modulation, the QKV projection with its per-head norm and 3-D RoPE, attention
(the forward call that keeps each row's log-sum-exp, and the backward call
that recomputes the probabilities from it), the gated out-projection and the
gated SwiGLU feed-forward.

A case names one operator and its sizes.  `run` computes it in elementary torch
operations in 32 bits, or with `own` set through the library's calls.  Packed
sequences are text, audio, video, padding to a multiple of 128 rows; outputs
over tokens come with their padding rows, which are zero.
"""
import math
import random

import torch

own = False

HEAD = 128
ROPE = (32, 48, 48)
THETA = 10000.0
EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# Widths of the trunk and of the small configuration of this repository.
FULL = {"D": 5376, "H": 56, "F": 14336}
TINY = {"D": 320, "H": 4, "F": 896}
RAGGED = {"D": 576, "H": 6, "F": 1280}
# Token counts (text, audio, video) of its workloads.
N_TINY = {"n_text": 16, "n_audio": 16, "n_video": 32}
N_RAGGED = {"n_text": 37, "n_audio": 58, "n_video": 240}
N_2S = {"n_text": 256, "n_audio": 160, "n_video": 7488}
N_5S = {"n_text": 512, "n_audio": 400, "n_video": 31248}
N_REFINER = {"n_text": 512, "n_audio": 0, "n_video": 0}


def listed():
    return [
        # AdaLN backward: the small configuration (launch latency), and the
        # residual gradient of a 768x1344 5 s sample (HBM streaming).
        {"name": "adaln_tiny", "op": "adaln", **TINY, **N_TINY, "branch": 0},
        {"name": "adaln_768x1344_5s", "op": "adaln", **FULL, **N_5S, "branch": 1},
        # QKV backward: ragged widths and lengths, and one 768x768 2 s sample.
        {"name": "qkv_ragged", "op": "qkv", **RAGGED, **N_RAGGED},
        {"name": "qkv_768sq_2s", "op": "qkv", **FULL, **N_2S},
        # Attention, forward and backward of one training pass: the small
        # configuration, a whole 768x768 2 s sample, and four heads (one of
        # fourteen sequence-parallel shares) of a 768x1344 5 s sample.
        {"name": "attention_tiny", "op": "attention", **TINY, **N_TINY},
        {"name": "attention_768sq_2s", "op": "attention", **FULL, **N_2S},
        {"name": "attention_768x1344_5s_4heads", "op": "attention", "D": 5376, "H": 4, "F": 14336, **N_5S},
        # Out-projection backward: the text refiner's 512 text tokens at full
        # width (few rows, whole weights), and a 768x1344 5 s sample.
        {"name": "out_refiner", "op": "out", **FULL, **N_REFINER},
        {"name": "out_768x1344_5s", "op": "out", **FULL, **N_5S},
        # Feed-forward backward: the small configuration, ragged widths and
        # lengths, and a 768x768 2 s sample at full width.
        {"name": "ffn_tiny", "op": "ffn", **TINY, **N_TINY},
        {"name": "ffn_ragged", "op": "ffn", **RAGGED, **N_RAGGED},
        {"name": "ffn_768sq_2s", "op": "ffn", **FULL, **N_2S},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adaln", "qkv", "attention", "out", "ffn"])
    D = 64 * _spread(rng, 3, 84)
    H = _spread(rng, 1, 56)
    F = 128 * _spread(rng, 2, 112)
    L = _spread(rng, 40, 32160)
    # no dearer than the largest listed case of the operator
    if op == "attention":
        L = min(L, int(math.sqrt(7904 ** 2 * 56 / H)))
    elif op == "ffn":
        L = min(L, max(40, 7904 * 5376 * 14336 // (D * F)))
    elif op == "qkv":
        L = min(L, max(40, 7904 * 5376 * 56 // (D * H)))
    share = [rng.random() if rng.random() < 0.85 else 0.0 for _ in range(3)]
    share[2] = max(share[2], 0.05)
    text = int(L * share[0] / sum(share))
    audio = int(L * share[1] / sum(share))
    case = {"op": op, "D": D, "H": H, "F": F, "n_text": text, "n_audio": audio, "n_video": L - text - audio}
    if op == "adaln":
        case["branch"] = rng.randrange(2)
    return case


def _sizes(case):
    L = case["n_text"] + case["n_audio"] + case["n_video"]
    return L, (L + 127) // 128 * 128


def _spans(case):
    """[start, end) rows of text, audio and video."""
    a = case["n_text"]
    b = a + case["n_audio"]
    return ((0, a), (a, b), (b, b + case["n_video"]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    L, Lp = _sizes(case)
    D, H, F = case["D"], case["H"], case["F"]
    I = H * HEAD

    def normal(*shape, std=1.0, mean=0.0, dtype=F32, rows=False):
        t = torch.empty(*shape, device="cuda", dtype=F32).normal_(mean, std, generator=g)
        if rows:  # token rows: the padding is zero
            t[L:] = 0
        return t.to(dtype)

    def heads(std=1.0):
        t = torch.empty(H, Lp, HEAD, device="cuda", dtype=F32).normal_(0.0, std, generator=g)
        t[:, L:] = 0
        return t

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("adaln", "out", "ffn"):
        s["mod"] = normal(3, 6, D, std=0.1)
    if op == "adaln":
        # the residual stream, with an offset and a scale as the trunk has it,
        # its gradient, and the gradient of the branch's input
        s["x"] = normal(Lp, D, std=3.0, mean=0.5, rows=True)
        s["dxm"] = normal(Lp, D, std=1e-3, dtype=BF16, rows=True)
        s["dres"] = normal(Lp, D, std=1e-3, rows=True)
    elif op == "qkv":
        s["xm"] = normal(Lp, D, dtype=BF16, rows=True)
        s["Wqkv"] = normal(3 * I, D, std=0.02, dtype=BF16)
        s["qn_w"] = normal(HEAD, std=0.1, mean=1.0, dtype=BF16)
        s["kn_w"] = normal(HEAD, std=0.1, mean=1.0, dtype=BF16)
        s["pos"] = _positions(case)
        for n in ("dq", "dk", "dv"):
            s[n] = heads(1e-3).to(BF16)
    elif op == "attention":
        # q and k as the QKV call leaves them: normalised rows times the norm weights
        s["qn_w"] = normal(HEAD, std=0.1, mean=1.0, dtype=BF16)
        s["kn_w"] = normal(HEAD, std=0.1, mean=1.0, dtype=BF16)
        for n in ("q", "k"):
            t = heads()
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * s[n + "n_w"].float()
            s[n] = t.to(BF16)
        s["v"] = heads().to(BF16)
        s["do"] = normal(Lp, I, std=1e-3, dtype=BF16, rows=True)
    elif op == "out":
        s["dx"] = normal(Lp, D, std=1e-3, rows=True)
        s["o"] = normal(Lp, I, std=0.3, dtype=BF16, rows=True)
        s["Wo"] = normal(D, I, std=0.02, dtype=BF16)
    else:
        s["dx"] = normal(Lp, D, std=1e-3, rows=True)
        s["xm"] = normal(Lp, D, dtype=BF16, rows=True)
        s["Wgu"] = normal(2 * F, D, std=0.02, dtype=BF16)
        s["Wd"] = normal(D, F, std=0.02, dtype=BF16)
    return s


def _positions(case):
    """(t, h, w) of every row: video over a grid 24 high and 42 wide, audio
    at 40 latents a second on the 6 Hz time axis, text and padding at 0."""
    _, Lp = _sizes(case)
    pos = torch.zeros(Lp, 3, device="cuda", dtype=F32)
    (_, a), (_, b), (_, e) = _spans(case)
    k = torch.arange(b - a, device="cuda")
    pos[a:b, 0] = (6 * k).float() / 40.0
    r = torch.arange(e - b, device="cuda")
    pos[b:e, 0] = (r // (24 * 42)).float()
    pos[b:e, 1] = (r // 42 % 24).float()
    pos[b:e, 2] = (r % 42).float()
    return pos


# ---------------------------------------------------------------- plain forms

def _rows_of(case, table):
    """One row of table [3][D] for every token."""
    n = torch.tensor([case["n_text"], case["n_audio"], case["n_video"]], device=table.device)
    return torch.repeat_interleave(table, n, dim=0)


def _sums(case, t):
    """Sums of t's token rows over each modality, [3][D]."""
    return torch.stack([t[a:b].sum(0) for a, b in _spans(case)])


def _pad(t, Lp, dtype):
    """Zero rows up to Lp (dimension -2)."""
    out = torch.zeros(*t.shape[:-2], Lp, t.shape[-1], device=t.device, dtype=dtype)
    out[..., :t.shape[-2], :] = t
    return out


def _rope_angles(pos):
    """Angle of every pair of a head, from 64-bit arithmetic."""
    parts = []
    for axis, d in enumerate(ROPE):
        f = THETA ** (-torch.arange(0, d, 2, device=pos.device, dtype=F64) / d)
        parts.append(pos[:, axis:axis + 1].double() * f)
    return torch.cat(parts, 1)


def _plain_adaln(s):
    case = s["case"]
    L, Lp = _sizes(case)
    b = 3 * case["branch"]
    x, dy = s["x"][:L], s["dxm"][:L].float()
    x = x - x.mean(1, keepdim=True)
    inv = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    xhat = x * inv
    dh = dy * (1 + _rows_of(case, s["mod"][:, b + 1]))
    dx = inv * (dh - dh.mean(1, keepdim=True) - xhat * (dh * xhat).mean(1, keepdim=True))
    return {"dx": _pad(s["dres"][:L] + dx, Lp, F32), "dshift": _sums(case, dy).to(BF16),
            "dscale": _sums(case, dy * xhat).to(BF16)}


def _plain_qkv(s):
    case = s["case"]
    L, Lp = _sizes(case)
    H = case["H"]
    I = H * HEAD
    xm, W = s["xm"][:L].float(), s["Wqkv"].float()
    angle = _rope_angles(s["pos"][:L])[:, None, :]
    cs, sn = angle.cos().float(), angle.sin().float()
    grads, norms = [], []
    raw = (xm @ W[:2 * I].T).view(L, 2, H, HEAD)
    for part, (dn, wn) in enumerate((("dq", "qn_w"), ("dk", "kn_w"))):
        d = s[dn][:, :L].float().transpose(0, 1)  # [L][H][128]
        even, odd = d[..., 0::2], d[..., 1::2]
        dy = torch.stack((even * cs + odd * sn, odd * cs - even * sn), -1).flatten(-2)  # turned back
        x = raw[:, part]
        inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xhat = x * inv
        norms.append((dy * xhat).sum((0, 1)).to(BF16))
        dh = dy * s[wn].float()
        grads.append(inv * (dh - xhat * (dh * xhat).mean(-1, keepdim=True)))
    grads.append(s["dv"][:, :L].float().transpose(0, 1))
    dqkv = torch.stack(grads, 1).reshape(L, 3 * I)
    return {"dxm": _pad(dqkv @ W, Lp, BF16), "dWqkv": (dqkv.T @ xm).to(BF16), "dqn_w": norms[0], "dkn_w": norms[1]}


def _plain_attention(s):
    case = s["case"]
    L, Lp = _sizes(case)
    H = case["H"]
    scale = 1.0 / math.sqrt(HEAD)
    q, k, v = (s[n][:, :L].float() for n in "qkv")
    do = s["do"][:L].float().view(L, H, HEAD).transpose(0, 1)
    p = torch.matmul(q, k.transpose(1, 2)).mul_(scale)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p.div_(total)
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(1, 2), do)
    ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(1, 2), q)
    return {"o": _pad(o.transpose(0, 1).reshape(L, H * HEAD), Lp, BF16), "lse": _pad(lse[..., None], Lp, F32)[..., 0],
            "dq": _pad(dq, Lp, BF16), "dk": _pad(dk, Lp, BF16), "dv": _pad(dv, Lp, BF16)}


def _plain_out(s):
    case = s["case"]
    L, Lp = _sizes(case)
    dx, o, W = s["dx"][:L], s["o"][:L].float(), s["Wo"].float()
    dy = dx * _rows_of(case, s["mod"][:, 2])
    return {"do": _pad(dy @ W, Lp, BF16), "dWo": (dy.T @ o).to(BF16), "dgate": _sums(case, dx * (o @ W.T)).to(BF16)}


def _plain_ffn(s):
    case = s["case"]
    L, Lp = _sizes(case)
    F = case["F"]
    dx, xm, Wgu, Wd = s["dx"][:L], s["xm"][:L].float(), s["Wgu"].float(), s["Wd"].float()
    gu = xm @ Wgu.T
    g, u = gu[:, :F], gu[:, F:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig
    h = act * u
    dy = dx * _rows_of(case, s["mod"][:, 5])
    dh = dy @ Wd
    dgu = torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * act), 1)
    return {"dxm": _pad(dgu @ Wgu, Lp, BF16), "dWgu": (dgu.T @ xm).to(BF16), "dWd": (dy.T @ h).to(BF16),
            "dgate": _sums(case, dx * (h @ Wd.T)).to(BF16)}


PLAIN = {"adaln": _plain_adaln, "qkv": _plain_qkv, "attention": _plain_attention, "out": _plain_out, "ffn": _plain_ffn}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from omni_modal_diffusion_b200 import h3

    case = s["case"]
    D, H, F = case["D"], case["H"], case["F"]
    I = H * HEAD
    dims = h3.make_dims(D, H, F, rope=ROPE, theta=THETA, eps_ln=EPS, eps_qk=EPS)
    r = h3.h3_make_ranges(case["n_text"], case["n_audio"], case["n_video"])
    Lp = r.L_pad

    def empty(*shape, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def workspace(op):
        return empty(h3.h3_backward_workspace_bytes(dims, Lp, op), dtype=torch.uint8)

    op = case["op"]
    if op == "adaln":
        dx, dmod = empty(Lp, D, dtype=F32), empty(3, 6, D)
        h3.h3_adaln_norm_modulate_backward(dims, r, s["x"], s["mod"], case["branch"], s["dxm"], s["dres"], dx, dmod,
                                           workspace(h3.H3_BWD_ADALN))
        b = 3 * case["branch"]
        return {"dx": dx, "dshift": dmod[:, b], "dscale": dmod[:, b + 1]}
    if op == "qkv":
        dxm, dW, dqn, dkn = empty(Lp, D), empty(3 * I, D), empty(HEAD), empty(HEAD)
        h3.h3_qkv_qknorm_mrope_backward(dims, r, s["xm"], s["Wqkv"], s["qn_w"], s["kn_w"], s["pos"], s["dq"], s["dk"],
                                        s["dv"], dxm, dW, dqn, dkn, workspace(h3.H3_BWD_QKV))
        return {"dxm": dxm, "dWqkv": dW, "dqn_w": dqn, "dkn_w": dkn}
    if op == "attention":
        o, lse = empty(Lp, I), empty(H, Lp, dtype=F32)
        dq, dk, dv = (empty(H, Lp, HEAD) for _ in range(3))
        h3.h3_attention_lse(dims, r, s["q"], s["k"], s["v"], o, lse, qn_w=s["qn_w"], kn_w=s["kn_w"])
        h3.h3_attention_backward(dims, r, s["q"], s["k"], s["v"], o, lse, s["do"], dq, dk, dv,
                                 workspace(h3.H3_BWD_ATTENTION))
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "out":
        do, dW, dmod = empty(Lp, I), empty(D, I), empty(3, 6, D)
        h3.h3_gated_residual_backward(dims, r, s["dx"], s["o"], s["Wo"], s["mod"], do, dW, dmod,
                                      workspace(h3.H3_BWD_GATED_RESIDUAL), branch=h3.H3_MSA)
        return {"do": do, "dWo": dW, "dgate": dmod[:, 2]}
    dxm, dWgu, dWd, dmod = empty(Lp, D), empty(2 * F, D), empty(D, F), empty(3, 6, D)
    h3.h3_ffn_swiglu_backward(dims, r, s["dx"], s["xm"], s["Wgu"], s["Wd"], s["mod"], dxm, dWgu, dWd, dmod,
                              workspace(h3.H3_BWD_FFN))
    return {"dxm": dxm, "dWgu": dWgu, "dWd": dWd, "dgate": dmod[:, 5]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    L, _ = _sizes(case)
    D, H, F, op = case["D"], case["H"], case["F"], case["op"]
    I = H * HEAD
    if op == "adaln":
        # x, the branch's gradient and the residual's in, the residual's out
        return {"bytes": L * D * (4 + 2 + 4 + 4) + 3 * D * (4 + 2 + 2), "flops": 16 * L * D}
    if op == "qkv":
        # q and k again, the input's gradient, the weight's
        return {"bytes": 2 * (2 * L * D + 3 * L * I + 6 * I * D) + 12 * L, "flops": 2 * L * D * I * (2 + 3 + 3)}
    if op == "attention":
        # forward: two products; backward: the scores again and four products
        return {"bytes": 2 * 8 * L * I + 4 * L * H, "flops": 2 * L * L * HEAD * H * (2 + 5)}
    if op == "out":
        return {"bytes": 4 * L * D + 2 * (2 * L * I + 2 * D * I) + 18 * D, "flops": 2 * L * D * I * 2}
    # gate and up again, the hidden state's gradient, the input's, the weights'
    return {"bytes": 4 * L * D + 2 * (2 * L * D + 6 * D * F) + 18 * D, "flops": 2 * L * D * F * (2 + 1 + 2 + 3)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """Each operator's definition in float64: the forward map is written down
    and its vector-Jacobian product taken by automatic differentiation, head by
    head where the probabilities of all heads would not fit."""
    s = prepare(case, seed)
    L, Lp = _sizes(case)
    D, H, F, op = case["D"], case["H"], case["F"], case["op"]
    spans = _spans(case)

    def leaf(t):
        return t.double().requires_grad_(True)

    def token_rows(t, width):
        return torch.cat((t, torch.zeros(Lp - L, width, device="cuda", dtype=F64)))

    if op == "adaln":
        x, shift, scale = leaf(s["x"][:L]), leaf(s["mod"][:, 3 * case["branch"]]), leaf(s["mod"][:, 3 * case["branch"] + 1])
        mu = x.mean(1, keepdim=True)
        xhat = (x - mu) / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + EPS)
        y = torch.cat([xhat[a:b] * (1 + scale[m]) + shift[m] for m, (a, b) in enumerate(spans)])
        y.backward(s["dxm"][:L].double())
        return {"dx": token_rows(x.grad + s["dres"][:L].double(), D), "dshift": shift.grad, "dscale": scale.grad}
    if op == "qkv":
        xm, W, qn, kn = leaf(s["xm"][:L]), leaf(s["Wqkv"]), leaf(s["qn_w"]), leaf(s["kn_w"])
        freq = [THETA ** (-2.0 * i / d) for d in ROPE for i in range(d // 2)]
        axis = [ax for ax, d in enumerate(ROPE) for _ in range(d // 2)]
        ang = s["pos"][:L].double()[:, axis] * torch.tensor(freq, device="cuda", dtype=F64)
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]
        q, k, v = (xm @ W.T).view(L, 3, H, HEAD).unbind(1)

        def place(t, w):
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * w
            return torch.view_as_real(torch.view_as_complex(t.reshape(L, H, HEAD // 2, 2)) * turn).reshape(L, H, HEAD)

        outs = [place(q, qn), place(k, kn), v]
        torch.autograd.backward(outs, [s[n][:, :L].double().transpose(0, 1) for n in ("dq", "dk", "dv")])
        return {"dxm": token_rows(xm.grad, D), "dWqkv": W.grad, "dqn_w": qn.grad, "dkn_w": kn.grad}
    if op == "attention":
        res = {n: torch.zeros(H, Lp, HEAD, device="cuda", dtype=F64) for n in ("dq", "dk", "dv")}
        o, lse = torch.zeros(Lp, H, HEAD, device="cuda", dtype=F64), torch.zeros(H, Lp, device="cuda", dtype=F64)
        do = s["do"].view(Lp, H, HEAD)
        for h in range(H):
            q, k, v, d = (t.double() for t in (s["q"][h, :L], s["k"][h, :L], s["v"][h, :L], do[:L, h]))
            w = q @ k.T / math.sqrt(HEAD)
            lse[h, :L] = torch.logsumexp(w, 1)
            w = torch.exp(w - lse[h, :L, None])
            o[:L, h] = w @ v
            res["dv"][h, :L] = w.T @ d
            w *= d @ v.T - (d * o[:L, h]).sum(1, keepdim=True)
            res["dq"][h, :L] = w @ k / math.sqrt(HEAD)
            res["dk"][h, :L] = w.T @ q / math.sqrt(HEAD)
        return {"o": o.view(Lp, H * HEAD), "lse": lse, **res}
    if op == "out":
        o, W, gate = leaf(s["o"][:L]), leaf(s["Wo"]), leaf(s["mod"][:, 2])
        y = o @ W.T
        y = torch.cat([y[a:b] * gate[m] for m, (a, b) in enumerate(spans)])
        y.backward(s["dx"][:L].double())
        return {"do": token_rows(o.grad, H * HEAD), "dWo": W.grad, "dgate": gate.grad}
    xm, Wgu, Wd, gate = leaf(s["xm"][:L]), leaf(s["Wgu"]), leaf(s["Wd"]), leaf(s["mod"][:, 5])
    g, u = xm @ Wgu[:F].T, xm @ Wgu[F:].T
    y = (g / (1 + torch.exp(-g)) * u) @ Wd.T
    y = torch.cat([y[a:b] * gate[m] for m, (a, b) in enumerate(spans)])
    y.backward(s["dx"][:L].double())
    return {"dxm": token_rows(xm.grad, D), "dWgu": Wgu.grad, "dWd": Wd.grad, "dgate": gate.grad}
