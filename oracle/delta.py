"""fp64 definition of the gated delta rule with one decay per head, token by token on the CPU (test infrastructure only,
like the rest of this package; it shares no code with the GPU path).

    S <- e^{g_t} S;   z_t = v_t - S^T k_t;   S <- S + beta_t k_t z_t^T;   o_t = scale S^T q_t

Its gradients by the chain rule through those lines, in reverse order of the tokens (G = dL/dS_t):
    G += scale q_t do_t^T;  dq_t = scale S_t do_t;  dw = G^T k_t;  dbeta_t = z_t.dw;  dv_t = beta_t dw;
    dk_t = beta_t G z_t - (e^g S_{t-1}) dv_t;  G -= k_t dv_t^T;  dg_t = <G, e^g S_{t-1}>;  G = e^g G.

``spread`` of either direction says how far a relative error of one part in every computed row may carry, by the triangle
inequality: with beta |k|^2 <= 2 each token's map of the state does not lengthen a column, so what a token adds to a
column's error stays as long as it is or decays.
"""
from __future__ import annotations

import torch

from .layers import F64, _expand, _seqs, f64


def _rows(q, k, v, g, beta, do=None):
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    n = B * T
    out = [_expand(f64(x).reshape(n, Hk, K), H) for x in (q, k)] + [f64(v).reshape(n, H, V)]
    out += [f64(x).reshape(n, H) for x in (g, beta)]
    return out + ([f64(do).reshape(n, H, V)] if do is not None else [])


def gd_forward(q, k, v, g, beta, S0=None, cu=None, scale=1.0, spread=False):
    """(o [B, T, H, V], S_final [N, H, K, V]); rows outside every sequence are NaN. With ``spread`` also those of o's
    entries and of S_final's columns [N, H, 1, V]."""
    B, T, _, K = q.shape
    H, V = v.shape[2:]
    q, k, v, g, beta = _rows(q, k, v, g, beta)
    o = torch.full((B * T, H, V), float("nan"), dtype=F64)
    so, ends, send = o.clone(), [], []
    for n, (t0, t1) in enumerate(_seqs(B, T, cu)):
        S = f64(S0)[n].clone() if S0 is not None else torch.zeros(H, K, V, dtype=F64)
        E = S.norm(dim=1)  # [H, V]
        for t in range(t0, t1):
            a = torch.exp(g[t])[:, None]
            S = a[..., None] * S
            z = v[t] - (k[t][:, :, None] * S).sum(1)
            E = a * E + beta[t][:, None].abs() * k[t].norm(dim=-1)[:, None] * (
                v[t].abs() + k[t].norm(dim=-1)[:, None] * S.norm(dim=1))
            S = S + (beta[t][:, None] * k[t])[:, :, None] * z[:, None, :]
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
            so[t] = abs(scale) * q[t].norm(dim=-1)[:, None] * (E + S.norm(dim=1))
        ends.append(S)
        send.append(E[:, None, :] + S.norm(dim=1, keepdim=True))
    res = o.reshape(B, T, H, V), torch.stack(ends)
    return (*res, so.reshape(B, T, H, V), torch.stack(send)) if spread else res


def gd_backward(q, k, v, g, beta, do, S0=None, dS=None, cu=None, scale=1.0, spread=False):
    """dict of dq, dk [B, T, Hk, K], dv [B, T, H, V], dg, dbeta [B, T, H], dS0. With ``spread`` also a dict of theirs."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k, v, g, beta, do = _rows(q, k, v, g, beta, do)
    nan = float("nan")
    sizes = {"dq": (K,), "dk": (K,), "dv": (V,), "dg": (), "dbeta": ()}
    out = {n: torch.full((B * T, H, *s), nan, dtype=F64) for n, s in sizes.items()}
    far = {n: x.clone() for n, x in out.items()}
    dS0, sdS0 = [], []
    sc = abs(scale)
    for n, (t0, t1) in enumerate(_seqs(B, T, cu)):
        states = [f64(S0)[n].clone() if S0 is not None else torch.zeros(H, K, V, dtype=F64)]
        errs = [states[0].norm(dim=1)]
        for t in range(t0, t1):
            a, kn = torch.exp(g[t])[:, None], k[t].norm(dim=-1)[:, None]
            S = a[..., None] * states[-1]
            z = v[t] - (k[t][:, :, None] * S).sum(1)
            errs.append(a * errs[-1] + beta[t][:, None].abs() * kn * (v[t].abs() + kn * S.norm(dim=1)))
            states.append(S + (beta[t][:, None] * k[t])[:, :, None] * z[:, None, :])
        G = f64(dS)[n].clone() if dS is not None else torch.zeros(H, K, V, dtype=F64)
        F = G.norm(dim=1)
        tail = (F * (errs[-1] + states[-1].norm(dim=1))).sum(-1)  # of dg: all that is summed behind a token
        for t in range(t1 - 1, t0 - 1, -1):
            a, b = torch.exp(g[t])[:, None, None], beta[t][:, None]
            qn, kn = q[t].norm(dim=-1)[:, None], k[t].norm(dim=-1)[:, None]
            S, before = states[t - t0 + 1], a * states[t - t0]
            E, Eb = errs[t - t0 + 1] + S.norm(dim=1), a[..., 0] * errs[t - t0] + before.norm(dim=1)
            G = G + scale * q[t][:, :, None] * do[t][:, None, :]
            F = F + sc * qn * do[t].abs()
            z = v[t] - (k[t][:, :, None] * before).sum(1)
            zs = v[t].abs() + kn * Eb  # how far z may carry
            dw = (G * k[t][:, :, None]).sum(1)
            ws = kn * (F + G.norm(dim=1))
            dv = b * dw
            out["dq"][t] = scale * (S * do[t][:, None, :]).sum(2)
            out["dbeta"][t] = (z * dw).sum(1)
            out["dv"][t] = dv
            out["dk"][t] = (G * (b * z)[:, None, :]).sum(2) - (before * dv[:, None, :]).sum(2)
            far["dq"][t] = sc * (E * do[t].abs()).sum(1)[:, None].expand(H, K)
            far["dbeta"][t] = (zs * ws).sum(1)
            far["dv"][t] = b.abs() * ws
            far["dk"][t] = (b.abs() * ((F + G.norm(dim=1)) * zs + Eb * ws)).sum(1)[:, None].expand(H, K)
            tail = tail + (sc * qn * E * do[t].abs() + b.abs() * (kn * Eb * ws + kn * zs * (F + G.norm(dim=1)))).sum(-1)
            far["dg"][t] = tail
            G = G - k[t][:, :, None] * dv[:, None, :]
            F = F + b.abs() * kn * ws
            out["dg"][t] = (G * before).sum((1, 2))
            G, F = a * G, a[..., 0] * F
        dS0.append(G)
        sdS0.append((F + G.norm(dim=1))[:, None, :].expand(H, K, V))

    def shape(x):
        r = {m: x[m].reshape(B, T, Hk, H // Hk, K).sum(3) for m in ("dq", "dk")}
        r.update(dv=x["dv"].reshape(B, T, H, V), dg=x["dg"].reshape(B, T, H), dbeta=x["dbeta"].reshape(B, T, H))
        return r

    res = {**shape(out), "dS0": torch.stack(dS0)}
    return (res, {**shape(far), "dS0": torch.stack(sdS0)}) if spread else res


def gd_step(q, k, v, g, beta, S, scale=1.0):
    """(o [N, H, V], S after the token)."""
    H = v.shape[1]
    q, k, v = _expand(f64(q), H), _expand(f64(k), H), f64(v)
    S = torch.exp(f64(g))[..., None, None] * f64(S)
    z = v - (k[..., None] * S).sum(2)
    S = S + (f64(beta)[..., None] * k)[..., None] * z[..., None, :]
    return scale * (q[..., None] * S).sum(2), S
