"""The gated delta rule with one decay per head: chunked forward, backward and single token.

Beside linear attention with one decay per head (layers.py) it corrects what the state already holds for a key; beside
KDA (chunk_fwd) its decay is one number per head instead of one per key channel, of any strength, and heads may share q
and k. Argument marshalling only, as in the rest of the package.
"""
from __future__ import annotations

import torch

from . import _io_code, _lib, _ptr
from .layers import _call, _cuda, _hd_seqs, _int32, _need, _restored, _result, _states, _workspace

__all__ = ["gd_chunk_fwd", "gd_chunk_bwd", "gd_decode_step", "gd_workspace_bytes", "gd_bwd_workspace_bytes"]


def gd_workspace_bytes(B: int, T: int, H: int, K: int, V: int, num_seqs: int, Hk: int = None, packed: bool = False,
                       io="bf16") -> int:
    """Device workspace bytes of gd_chunk_fwd (0 = unsupported sizes)."""
    return int(_lib.load().kda_gd_chunk_fwd_workspace_bytes(B, T, H, H if Hk is None else Hk, K, V, num_seqs,
                                                            int(bool(packed)), _io_code(io)))


def gd_bwd_workspace_bytes(B: int, T: int, H: int, K: int, V: int, num_seqs: int, Hk: int = None,
                           packed: bool = False, io="bf16") -> int:
    """Device workspace bytes of gd_chunk_bwd (0 = unsupported sizes)."""
    return int(_lib.load().kda_gd_chunk_bwd_workspace_bytes(B, T, H, H if Hk is None else Hk, K, V, num_seqs,
                                                            int(bool(packed)), _io_code(io)))


def _inputs(q, k, v, g, beta, lead):
    """Checks q, k [*lead, Hk, K], v [*lead, H, V], g and beta [*lead, H]; returns (H, Hk, K, V, dtype, gates' code)."""
    dev, dt = q.device, q.dtype
    Hk, K = q.shape[-2:]
    if v.dim() != len(lead) + 2:
        raise ValueError("v has shape %s, expected %d dimensions" % (tuple(v.shape), len(lead) + 2))
    H, V = v.shape[-2:]
    if Hk < 1 or H % Hk:
        raise ValueError("v's %d heads are no whole multiple of q's %d" % (H, Hk))
    _need(q, "q", lead + (Hk, K), dt, dev)
    _need(k, "k", lead + (Hk, K), dt, dev)
    _need(v, "v", lead + (H, V), dt, dev)
    if (H * V | Hk * K) >> 31:
        _int32(H, Hk, K, V)
    gt = torch.float32 if g.dtype is torch.float32 else dt
    _need(g, "g", lead + (H,), gt, dev)
    _need(beta, "beta", lead + (H,), gt, dev)
    return H, Hk, K, V, dt, _io_code(gt)


def gd_chunk_fwd(q, k, v, g, beta, S0=None, cu_seqlens=None, scale: float = 1.0, output_final_state: bool = True,
                 workspace=None, out=None, final_state_out=None):
    """The gated delta rule with one decay per head over whole sequences: S <- exp(g_t) S, then
    S <- S + beta_t k_t (v_t - S^T k_t)^T, o_t = scale S^T q_t. Returns (o, S_final or None).

    q, k [B, T, Hk, K]; v [B, T, H, V] with H a whole multiple of Hk (head h reads q/k head h // (H // Hk)); K and V
    of 32, 64 or 128; bf16 or fp32. ``g`` (the log-decay, at most 0 in use; -inf clears the state) and ``beta`` are
    [B, T, H], both in the input dtype or both fp32. The rule contracts where beta |k|^2 <= 2: give keys of length one
    (layer_norm_fwd without centering and weights K^-1/2 makes them). S0 and S_final are fp32 [num_seqs, H, K, V]. With
    ``cu_seqlens`` (int32 [num_seqs + 1], on the device) B must be 1 and the sequences are packed along T; rows of
    ``out`` outside them are left as they are. ``workspace`` (uint8, gd_workspace_bytes()), ``out`` and
    ``final_state_out`` may be passed to avoid allocations.
    """
    lib = _lib.load()
    dev = _cuda(q)
    N = _hd_seqs(q, cu_seqlens)
    B, T = q.shape[:2]
    H, Hk, K, V, dt, gates = _inputs(q, k, v, g, beta, (B, T))
    io = _io_code(dt)
    if S0 is not None:
        _need(S0, "S0", (N, H, K, V), torch.float32, dev)
    need = lib.kda_gd_chunk_fwd_workspace_bytes(B, T, H, Hk, K, V, N, int(cu_seqlens is not None), io)
    workspace = _workspace(workspace, need, dev, "gd_chunk_fwd(B=%d, T=%d, H=%d, Hk=%d, K=%d, V=%d, num_seqs=%d)",
                           B, T, H, Hk, K, V, N)
    out = _result(out, "out", v)
    S = None
    if final_state_out is not None or output_final_state:
        S = _states(final_state_out, "final_state_out", S0, (N, H, K, V), dev)
    _call(dev, lib.kda_gd_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens), B, T,
          H, Hk, K, V, N, io, gates, scale, _ptr(out), _ptr(S), _ptr(workspace), workspace.numel())
    return out, S


def gd_chunk_bwd(q, k, v, g, beta, do, S0=None, dS_final=None, cu_seqlens=None, scale: float = 1.0,
                 want_dS0: bool = True, workspace=None, out=None):
    """Gradients of gd_chunk_fwd's (o, S_final) given ``do`` = dL/do (o's shape, input dtype) and ``dS_final`` (fp32
    [num_seqs, H, K, V], or None: zero). Returns a dict: dq, dk, dv in the inputs' shapes and dtype (dq and dk summed
    over the heads that share them); dg and dbeta like g and beta; dS0 fp32 when ``want_dS0``. ``out`` may hold
    preallocated results by these names. Nothing of a forward call is needed; deterministic. q, k and v may each be a
    Checkpoint8: it is restored to a tensor that the call allocates, whatever is preallocated.
    """
    lib = _lib.load()
    q, k, v = _restored(q, k, v)
    dev = _cuda(q)
    N = _hd_seqs(q, cu_seqlens)
    B, T = q.shape[:2]
    H, Hk, K, V, dt, gates = _inputs(q, k, v, g, beta, (B, T))
    io = _io_code(dt)
    _need(do, "do", (B, T, H, V), dt, dev)
    for name, t in (("S0", S0), ("dS_final", dS_final)):
        if t is not None:
            _need(t, name, (N, H, K, V), torch.float32, dev)
    like = {"dq": q, "dk": k, "dv": v, "dg": g, "dbeta": beta}
    given = out or {}
    for name in given:
        if name not in like and not (name == "dS0" and want_dS0):
            raise ValueError("out[%r]: not a result of this call" % (name,))
    need = lib.kda_gd_chunk_bwd_workspace_bytes(B, T, H, Hk, K, V, N, int(cu_seqlens is not None), io)
    workspace = _workspace(workspace, need, dev, "gd_chunk_bwd(B=%d, T=%d, H=%d, Hk=%d, K=%d, V=%d, num_seqs=%d)",
                           B, T, H, Hk, K, V, N)
    res = {n: _result(given.get(n), n, t) for n, t in like.items()}
    if want_dS0:
        res["dS0"] = _states(given.get("dS0"), "dS0", S0 if S0 is not None else dS_final, (N, H, K, V), dev)
    _call(dev, lib.kda_gd_chunk_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
          _ptr(do), _ptr(dS_final), B, T, H, Hk, K, V, N, io, gates, scale, _ptr(res["dq"]), _ptr(res["dk"]),
          _ptr(res["dv"]), _ptr(res["dg"]), _ptr(res["dbeta"]), _ptr(res.get("dS0")), _ptr(workspace),
          workspace.numel())
    return res


def gd_decode_step(q, k, v, g, beta, S, scale: float = 1.0, out=None):
    """One token of every sequence: q, k [N, Hk, K], v [N, H, V], g and beta [N, H] (both in the input dtype or both
    fp32); S [N, H, K, V] fp32 is updated in place. Returns o [N, H, V] in the input dtype."""
    lib = _lib.load()
    dev = _cuda(q)
    if q.dim() != 3:
        raise ValueError("q has shape %s, expected [N, heads, K]" % (tuple(q.shape),))
    N = q.shape[0]
    H, Hk, K, V, dt, gates = _inputs(q, k, v, g, beta, (N,))
    _need(S, "S", (N, H, K, V), torch.float32, dev)
    out = _result(out, "out", v)
    _call(dev, lib.kda_gd_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(out), N, H, Hk, K,
          V, _io_code(dt), gates, scale)
    return out
