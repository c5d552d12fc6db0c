"""fp64 definitions of the operators around the recurrence, token by token on the CPU (test infrastructure only, like
the rest of this package; it shares no code with the GPU path).

Linear attention with one decay per head:  S <- e^{g_t} S + k_t v_t^T,  o_t = scale S^T q_t.
Its gradients by the chain rule through those two lines, in reverse order of the tokens (G = dL/dS_t):
  G += scale q_t do_t^T;  dq_t = scale S_t do_t;  dk_t = G v_t;  dv_t = G^T k_t;  dg_t = <G, e^{g_t} S_{t-1}>;
  G = e^{g_t} G.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def f64(x):
    return None if x is None else x.detach().to("cpu", F64)


def _expand(x, H):
    """[T, Hk, D] -> [T, H, D]: head h reads h // (H / Hk)."""
    return x.repeat_interleave(H // x.shape[1], dim=1)


def _seqs(B, T, cu):
    """(first token, last token + 1) of every sequence in the flattened rows, as the library reads cu_seqlens."""
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    top, edges = 0, []
    for x in cu.tolist():
        top = max(top, min(max(int(x), 0), T))
        edges.append(top)
    return list(zip(edges[:-1], edges[1:]))


def hd_forward(q, k, v, g, S0=None, cu=None, scale=1.0):
    """(o [B, T, H, V], S_final [N, H, K, V]); rows outside every sequence are NaN."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k = (_expand(f64(x).reshape(B * T, Hk, K), H) for x in (q, k))
    v = f64(v).reshape(B * T, H, V)
    a = torch.exp(f64(g)).expand(B * T, H) if g.dim() == 1 else torch.exp(f64(g)).reshape(B * T, H)
    o = torch.full((B * T, H, V), float("nan"), dtype=F64)
    ends = []
    for n, (t0, t1) in enumerate(_seqs(B, T, cu)):
        S = f64(S0)[n].clone() if S0 is not None else torch.zeros(H, K, V, dtype=F64)
        for t in range(t0, t1):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
        ends.append(S)
    return o.reshape(B, T, H, V), torch.stack(ends)


def hd_backward(q, k, v, g, do, S0=None, dS=None, cu=None, scale=1.0):
    """dict of dq, dk [B, T, Hk, K], dv [B, T, H, V], dg [B, T, H] (also for g per head: per token), dS0."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    qe, ke = (_expand(f64(x).reshape(B * T, Hk, K), H) for x in (q, k))
    v, do = f64(v).reshape(B * T, H, V), f64(do).reshape(B * T, H, V)
    a = torch.exp(f64(g)).expand(B * T, H) if g.dim() == 1 else torch.exp(f64(g)).reshape(B * T, H)
    nan = float("nan")
    dq, dk = (torch.full((B * T, H, K), nan, dtype=F64) for _ in range(2))
    dv, dg = torch.full((B * T, H, V), nan, dtype=F64), torch.full((B * T, H), nan, dtype=F64)
    dS0 = []
    for n, (t0, t1) in enumerate(_seqs(B, T, cu)):
        states = [f64(S0)[n].clone() if S0 is not None else torch.zeros(H, K, V, dtype=F64)]
        for t in range(t0, t1):
            states.append(a[t][:, None, None] * states[-1] + ke[t][:, :, None] * v[t][:, None, :])
        G = f64(dS)[n].clone() if dS is not None else torch.zeros(H, K, V, dtype=F64)
        for t in range(t1 - 1, t0 - 1, -1):
            S, before = states[t - t0 + 1], states[t - t0]
            G = G + scale * qe[t][:, :, None] * do[t][:, None, :]
            dq[t] = scale * (S * do[t][:, None, :]).sum(2)
            dk[t] = (G * v[t][:, None, :]).sum(2)
            dv[t] = (G * ke[t][:, :, None]).sum(1)
            dg[t] = a[t] * (G * before).sum((1, 2))
            G = a[t][:, None, None] * G
        dS0.append(G)
    group = H // Hk
    return {"dq": dq.reshape(B, T, Hk, group, K).sum(3), "dk": dk.reshape(B, T, Hk, group, K).sum(3),
            "dv": dv.reshape(B, T, H, V), "dg": dg.reshape(B, T, H), "dS0": torch.stack(dS0)}


def hd_step(q, k, v, g, S, scale=1.0):
    """(o [N, H, V], S after the token)."""
    H = v.shape[1]
    q, k, v = _expand(f64(q), H), _expand(f64(k), H), f64(v)
    S = torch.exp(f64(g)).expand(v.shape[0], H)[..., None, None] * f64(S) + k[..., :, None] * v[..., None, :]
    return scale * (q[..., :, None] * S).sum(2), S


def rotate(x, freqs, positions, layout="half", inverse=False, scale=1.0):
    """x [..., heads, D] with positions of its leading shape."""
    angle = f64(positions)[..., None] * f64(freqs) * (-1.0 if inverse else 1.0)
    turn = torch.polar(torch.full_like(angle, scale), angle)[..., None, :]
    y, R = f64(x).clone(), 2 * freqs.numel()
    first, second = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def norm_forward(x, w=None, b=None, z=None, eps=1e-5, center=True):
    x = f64(x)
    if center:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = y * (f64(w) if w is not None else 1.0) + (f64(b) if b is not None else 0.0)
    return y * torch.sigmoid(f64(z)) if z is not None else y


def norm_backward(dy, x, w=None, b=None, z=None, eps=1e-5, center=True):
    """dict of dx, dweight, dbias, do_gate (where w, b, z are given), parameters summed over the rows."""
    x, dy = f64(x), f64(dy)
    C = x.shape[-1]
    xc = x - x.mean(-1, keepdim=True) if center else x
    r = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    n = xc * r
    out = {}
    if z is not None:
        a = torch.sigmoid(f64(z))
        out["do_gate"] = dy * (n * (f64(w) if w is not None else 1.0) + (f64(b) if b is not None else 0.0)) * a * (1 - a)
        dy = dy * a
    for name, p, e in (("dweight", w, dy * n), ("dbias", b, dy)):
        if p is not None:
            out[name] = e.reshape(-1, *p.shape).sum(0)
    d = dy * (f64(w) if w is not None else 1.0)
    # n_i depends on every x_j: dn_i/dx_j = r (delta_ij - 1/C [centered] - n_i n_j / C)
    dx = d - n * (d * n).sum(-1, keepdim=True) / C
    if center:
        dx = dx - d.sum(-1, keepdim=True) / C
    out["dx"] = r * dx
    return out


def rotate_axes(x, freqs, axes, positions, layout="half", inverse=False, scale=1.0):
    """rotate() with several axes, pair by pair: pair j turns by positions[axes[j]]."""
    y, P = f64(x).clone(), freqs.numel()
    for j in range(P):
        angle = f64(positions)[int(axes[j])][..., None] * f64(freqs)[j] * (-1.0 if inverse else 1.0)
        one, two = (j, j + P) if layout == "half" else (2 * j, 2 * j + 1)
        a, b = f64(x)[..., one], f64(x)[..., two]
        y[..., one] = scale * (a * torch.cos(angle) - b * torch.sin(angle))
        y[..., two] = scale * (a * torch.sin(angle) + b * torch.cos(angle))
    return y


def save8(x):
    """(codes, scales) of a checkpoint in 8 bits, block by block: the exact quotients are formed in whole numbers where
    they could be a tie (127 x is exact in fp64)."""
    x = f64(x)
    codes, scales = torch.zeros_like(x), []
    for c in range(0, x.shape[-1], 128):
        b = x[..., c:c + 128]
        top = b.abs().amax(-1, keepdim=True)
        codes[..., c:c + 128] = torch.where(top > 0, torch.round(127 * b / top.clamp(min=1e-300)), 0.0)
        scales.append(top / 127)
    return codes.to(torch.int8), torch.cat(scales, -1)


def restore8(codes, scales):
    """The values in fp64, unrounded."""
    x = f64(codes)
    for i in range(scales.shape[-1]):
        x[..., 128 * i:128 * i + 128] *= f64(scales)[..., i, None]
    return x
