"""The operators around the recurrence: linear attention with one decay per head (chunked forward, backward, single
token), rotary positions with one or several axes, layer norm and its gradient, activation checkpoints in 8 bits.

Like the rest of the package this only marshals tensors into libkda.so: it checks shapes, dtypes and devices,
allocates outputs and workspaces with torch, and passes pointers and torch's current stream of the tensors' device.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import KDAError, _io_code, _lib, _ptr
from . import _need as _explain

__all__ = ["hd_chunk_fwd", "hd_chunk_bwd", "hd_decode_step", "hd_workspace_bytes", "hd_bwd_workspace_bytes", "rotary",
           "rotary_freqs", "rotary_axes", "rotary_sections", "layer_norm_fwd", "layer_norm_bwd", "Checkpoint8",
           "checkpoint8", "restore8"]


# the current stream's handle by device index, without making a Stream object of it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(dev, fn, *args) -> None:
    """fn(*args, stream) on dev's current stream, with dev current while the kernels are enqueued."""
    i = dev.index
    if i == torch.cuda.current_device():
        status = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(i))
    if status:
        raise KDAError(status, fn.__name__)


def _need(t, name, shape, dtype, dev):
    """The package's check of an argument; what is right passes on one line (small calls cost little else)."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        _explain(t, name, shape, dtype, dev)


def _cuda(t):
    if t.device.type != "cuda":
        raise ValueError("inputs must be CUDA (HIP) tensors")
    return t.device


def _int32(*sizes):
    """Sizes that go into the library as 32-bit numbers: ctypes would pass on the low bits of larger ones."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("sizes %s: at most 2^31 - 1" % (sizes,))


def _workspace(workspace, need: int, dev, what: str, *sizes):
    if need == 0:
        raise KDAError(2, what % sizes)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    return workspace


_untouched = {}


def _no_workspace(dev):
    """What a call that keeps nothing in its workspace is given: any calls may name the same bytes."""
    if dev not in _untouched:
        _untouched[dev] = torch.empty(256, dtype=torch.uint8, device=dev)
    return _untouched[dev]


def _result(out, name, like):
    """The caller's tensor for a result of ``like``'s shape, dtype and device, or a new one."""
    if out is None:
        return torch.empty_like(like)
    _need(out, name, like.shape, like.dtype, like.device)
    return out


def _states(out, name, S, shape, dev):
    """The same for the states [num_seqs, H, K, V], like S where there is one."""
    if out is None:
        return torch.empty(shape, dtype=torch.float32, device=dev) if S is None else torch.empty_like(S)
    _need(out, name, shape, torch.float32, dev)
    return out


# ---------------------------------------------------------------- activation checkpoints in 8 bits
class Checkpoint8(NamedTuple):
    """A tensor of ``dtype`` in 8 bits: int8 ``codes`` of its shape, and an fp32 scale for 128 adjacent values of its
    last axis, [..., ceil(C / 128)]. It stands for codes * scales, rounded to ``dtype``. The backward passes that say so
    take it in place of the tensor."""
    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype


def _blocks8(shape):
    return (*shape[:-1], (shape[-1] + 127) // 128)


def _need8(c, name, shape, dev):
    _need(c.codes, name + ".codes", shape, torch.int8, dev)
    _need(c.scales, name + ".scales", _blocks8(shape), torch.float32, dev)


def checkpoint8(x, out=None):
    """x [..., C] (bf16 or fp32) as a Checkpoint8: codes = 127 x / max |x| to the nearest whole number (ties to even),
    scales = max |x| / 127, the maximum over 128 adjacent values of the last axis. Before it is rounded to x's dtype a
    value is off by at most half a scale; a block with an infinity or a NaN comes back as NaN. ``out`` may hold a
    Checkpoint8 to write into."""
    lib = _lib.load()
    dev, io = _cuda(x), _io_code(x.dtype)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x has shape %s, expected at least one value in a row" % (tuple(x.shape),))
    _int32(x.shape[-1])
    _need(x, "x", x.shape, x.dtype, dev)
    if out is None:
        out = Checkpoint8(torch.empty(x.shape, dtype=torch.int8, device=dev),
                          torch.empty(_blocks8(x.shape), dtype=torch.float32, device=dev), x.dtype)
    else:
        _need8(out, "out", x.shape, dev)
        if out.dtype is not x.dtype:
            raise TypeError("out.dtype is %s, expected %s" % (out.dtype, x.dtype))
    _call(dev, lib.kda_checkpoint8_save, _ptr(x), _ptr(out.codes), _ptr(out.scales), math.prod(x.shape[:-1]),
          x.shape[-1], io)
    return out


def restore8(c, out=None):
    """The tensor that the Checkpoint8 ``c`` stands for."""
    lib = _lib.load()
    dev, io, shape = _cuda(c.codes), _io_code(c.dtype), c.codes.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("codes has shape %s, expected at least one value in a row" % (tuple(shape),))
    _int32(shape[-1])
    _need8(c, "c", shape, dev)
    if out is None:
        out = torch.empty(shape, dtype=c.dtype, device=dev)
    else:
        _need(out, "out", shape, c.dtype, dev)
    _call(dev, lib.kda_checkpoint8_restore, _ptr(c.codes), _ptr(c.scales), _ptr(out), math.prod(shape[:-1]), shape[-1],
          io)
    return out


def _restored(*tensors):
    """The tensors as they are, checkpoints restored."""
    return tuple(restore8(t) if isinstance(t, Checkpoint8) else t for t in tensors)


# ---------------------------------------------------------------- linear attention with one decay per head
def hd_workspace_bytes(B: int, T: int, H: int, K: int, V: int, num_seqs: int, Hk: int = None, packed: bool = False,
                       io="bf16") -> int:
    """Device workspace bytes of hd_chunk_fwd (0 = unsupported sizes)."""
    return int(_lib.load().kda_hd_chunk_fwd_workspace_bytes(B, T, H, H if Hk is None else Hk, K, V, num_seqs,
                                                            int(bool(packed)), _io_code(io)))


def hd_bwd_workspace_bytes(B: int, T: int, H: int, K: int, V: int, num_seqs: int, Hk: int = None,
                           packed: bool = False, io="bf16") -> int:
    """Device workspace bytes of hd_chunk_bwd (0 = unsupported sizes)."""
    return int(_lib.load().kda_hd_chunk_bwd_workspace_bytes(B, T, H, H if Hk is None else Hk, K, V, num_seqs,
                                                            int(bool(packed)), _io_code(io)))


def _hd_inputs(q, k, v, g, lead):
    """Checks q, k [*lead, Hk, K], v [*lead, H, V] and g; returns (H, Hk, K, V, dtype, decay code)."""
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
    if g.dim() == 1:
        _need(g, "g", (H,), torch.float32, dev)
        return H, Hk, K, V, dt, _lib.KDA_DECAY_PER_HEAD
    _need(g, "g", lead + (H,), dt, dev)
    return H, Hk, K, V, dt, _lib.KDA_DECAY_PER_TOKEN


def _hd_seqs(q, cu_seqlens):
    if q.dim() != 4:
        raise ValueError("q has shape %s, expected [B, T, heads, K]" % (tuple(q.shape),))
    if cu_seqlens is None:
        return q.shape[0]
    _need(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, q.device)
    _int32(cu_seqlens.numel())
    return cu_seqlens.numel() - 1


def hd_chunk_fwd(q, k, v, g, S0=None, cu_seqlens=None, scale: float = 1.0, output_final_state: bool = True,
                 workspace=None, out=None, final_state_out=None):
    """Linear attention with one decay per head over whole sequences: S <- exp(g_t) S + k_t v_t^T,
    o_t = scale S^T q_t. Returns (o, S_final or None).

    q, k [B, T, Hk, K]; v [B, T, H, V] with H a whole multiple of Hk (head h reads q/k head h // (H // Hk)); K and V
    of 32, 64 or 128; bf16 or fp32. ``g`` is the log-decay: [B, T, H] in the input dtype, or [H] fp32, a constant of
    each head. At most 0 in use; -inf clears the state. S0 and S_final are fp32 [num_seqs, H, K, V]. With
    ``cu_seqlens`` (int32 [num_seqs + 1], on the device) B must be 1 and the sequences are packed along T; rows of
    ``out`` outside them are left as they are. ``workspace`` (uint8, hd_workspace_bytes()), ``out`` and
    ``final_state_out`` may be passed to avoid allocations.
    """
    lib = _lib.load()
    dev = _cuda(q)
    N = _hd_seqs(q, cu_seqlens)
    B, T = q.shape[:2]
    H, Hk, K, V, dt, decay = _hd_inputs(q, k, v, g, (B, T))
    io = _io_code(dt)
    if S0 is not None:
        _need(S0, "S0", (N, H, K, V), torch.float32, dev)
    need = lib.kda_hd_chunk_fwd_workspace_bytes(B, T, H, Hk, K, V, N, int(cu_seqlens is not None), io)
    if workspace is None and need == 256:
        workspace = _no_workspace(dev)
    workspace = _workspace(workspace, need, dev, "hd_chunk_fwd(B=%d, T=%d, H=%d, Hk=%d, K=%d, V=%d, num_seqs=%d)",
                           B, T, H, Hk, K, V, N)
    out = _result(out, "out", v)
    S = None
    if final_state_out is not None or output_final_state:
        S = _states(final_state_out, "final_state_out", S0, (N, H, K, V), dev)
    _call(dev, lib.kda_hd_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(cu_seqlens), B, T, H, Hk, K, V,
          N, io, decay, scale, _ptr(out), _ptr(S), _ptr(workspace), workspace.numel())
    return out, S


def hd_chunk_bwd(q, k, v, g, do, S0=None, dS_final=None, cu_seqlens=None, scale: float = 1.0, want_dS0: bool = True,
                 want_dg: bool = True, workspace=None, out=None):
    """Gradients of hd_chunk_fwd's (o, S_final) given ``do`` = dL/do (o's shape, input dtype) and ``dS_final`` (fp32
    [num_seqs, H, K, V], or None: zero). Returns a dict: dq, dk, dv in the inputs' shapes and dtype (dq and dk summed
    over the heads that share them); dg [B, T, H] when g is per token and ``want_dg`` (a constant per head has no
    gradient here: give it per token and sum); dS0 fp32 when ``want_dS0``. ``out`` may hold preallocated results by
    these names. Nothing of a forward call is needed; deterministic. q, k and v may each be a Checkpoint8: it is
    restored to a tensor that the call allocates, whatever is preallocated.
    """
    lib = _lib.load()
    q, k, v = _restored(q, k, v)
    dev = _cuda(q)
    N = _hd_seqs(q, cu_seqlens)
    B, T = q.shape[:2]
    H, Hk, K, V, dt, decay = _hd_inputs(q, k, v, g, (B, T))
    io = _io_code(dt)
    _need(do, "do", (B, T, H, V), dt, dev)
    for name, t in (("S0", S0), ("dS_final", dS_final)):
        if t is not None:
            _need(t, name, (N, H, K, V), torch.float32, dev)
    like = {"dq": q, "dk": k, "dv": v}
    if want_dg and decay == _lib.KDA_DECAY_PER_TOKEN:
        like["dg"] = g
    given = out or {}
    for name in given:
        if name not in like and not (name == "dS0" and want_dS0):
            raise ValueError("out[%r]: not a result of this call" % (name,))
    need = lib.kda_hd_chunk_bwd_workspace_bytes(B, T, H, Hk, K, V, N, int(cu_seqlens is not None), io)
    workspace = _workspace(workspace, need, dev, "hd_chunk_bwd(B=%d, T=%d, H=%d, Hk=%d, K=%d, V=%d, num_seqs=%d)",
                           B, T, H, Hk, K, V, N)
    res = {n: _result(given.get(n), n, t) for n, t in like.items()}
    if want_dS0:
        res["dS0"] = _states(given.get("dS0"), "dS0", S0 if S0 is not None else dS_final, (N, H, K, V), dev)
    _call(dev, lib.kda_hd_chunk_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(cu_seqlens), _ptr(do),
          _ptr(dS_final), B, T, H, Hk, K, V, N, io, decay, scale, _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]),
          _ptr(res.get("dg")), _ptr(res.get("dS0")), _ptr(workspace), workspace.numel())
    return res


def hd_decode_step(q, k, v, g, S, scale: float = 1.0, out=None):
    """One token of every sequence: q, k [N, Hk, K], v [N, H, V], g [N, H] (input dtype) or [H] (fp32); S
    [N, H, K, V] fp32 is updated in place. Returns o [N, H, V] in the input dtype."""
    lib = _lib.load()
    dev = _cuda(q)
    if q.dim() != 3:
        raise ValueError("q has shape %s, expected [N, heads, K]" % (tuple(q.shape),))
    N = q.shape[0]
    H, Hk, K, V, dt, decay = _hd_inputs(q, k, v, g, (N,))
    io = _io_code(dt)
    _need(S, "S", (N, H, K, V), torch.float32, dev)
    out = _result(out, "out", v)
    _call(dev, lib.kda_hd_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S), _ptr(out), N, H, Hk, K, V, io,
          decay, scale)
    return out


# ---------------------------------------------------------------- rotary positions
def rotary_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_context: int = None, low: float = 1.0, high: float = 32.0, device="cuda"):
    """Angular frequencies (radians per position) of the rot_dim / 2 channel pairs, fp64 on ``device``:
    base^(-2j / rot_dim), for contexts ``factor`` times the trained one stretched by ``scaling``:

    "none"      as they are;
    "linear"    all divided by ``factor`` (positions interpolated);
    "by_parts"  by how many turns a pair makes over ``original_context`` tokens: pairs of ``high`` turns or more stay,
                pairs of ``low`` turns or fewer are divided by ``factor``, those between blend linearly.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if not original_context or not high > low:
            raise ValueError("by_parts needs original_context and high > low")
        turns = original_context * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling != "none":
        raise ValueError("scaling must be one of ['by_parts', 'linear', 'none']")
    return f.to(device)


def rotary(q, freqs, k=None, positions=None, layout: str = "half", inverse: bool = False, scale: float = 1.0, out=None,
           k_out=None):
    """Rotary positions: turns the first 2 * len(freqs) channels of every head of q [..., Hq, D] (and k [..., Hk, D])
    in pairs j by the angle position * freqs[j] and copies the others. Returns the turned q, or (q, k).

    ``layout``: "half" pairs (j, j + len(freqs)), "interleaved" pairs (2j, 2j + 1). ``freqs``: fp64 (rotary_freqs());
    angles are exact at any int32 position, a frequency that is not finite makes its pair NaN. ``positions``: int32 of
    q's leading shape; None counts 0 .. T-1 along the third axis from the end. ``scale`` multiplies the turned channels.
    ``inverse`` turns back: the gradient of the same call without it. ``out`` / ``k_out`` may be q / k themselves (in
    place).
    """
    lib = _lib.load()
    dev = _cuda(q)
    if layout not in _lib.ROTARY_LAYOUTS:
        raise ValueError("layout must be one of %s" % sorted(_lib.ROTARY_LAYOUTS))
    if q.dim() < 3:
        raise ValueError("q has shape %s, expected [..., heads, channels]" % (tuple(q.shape),))
    lead, (Hq, D), dt = q.shape[:-2], q.shape[-2:], q.dtype
    io = _io_code(dt)
    _need(q, "q", q.shape, dt, dev)
    _need(freqs, "freqs", (freqs.numel(),), torch.float64, dev)
    Hk = 0
    if k is not None:
        Hk = k.shape[-2] if k.dim() == q.dim() else -1
        _need(k, "k", lead + (Hk, D), dt, dev)
        k_out = _result(k_out, "k_out", k)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if positions is not None:
        _need(positions, "positions", lead, torch.int32, dev)
    if ((Hq + Hk) * D + freqs.numel()) >> 30:
        _int32(Hq, Hk, D, 2 * freqs.numel())
    out = _result(out, "out", q)
    _call(dev, lib.kda_rotary, _ptr(q), _ptr(k), _ptr(freqs), _ptr(positions), _ptr(out), _ptr(k_out),
          math.prod(lead), lead[-1], Hq, Hk, D, 2 * freqs.numel(), io, _lib.ROTARY_LAYOUTS[layout], int(bool(inverse)),
          scale)
    return out if k is None else (out, k_out)


def rotary_sections(sections, order: str = "runs", device="cuda"):
    """The axis of every channel pair, int32 on ``device``, for rotary_axes: sections[a] pairs turn by axis a, in ``order``
    "runs" (axis 0's pairs first, then axis 1's, ...) or "turns" (a pair of each axis in turn while it has any left)."""
    left = [int(n) for n in sections]
    if order not in ("runs", "turns"):
        raise ValueError("order must be one of ['runs', 'turns']")
    if not left or min(left) < 0 or sum(left) < 1:
        raise ValueError("sections must be counts of pairs, one at least")
    axes = []
    if order == "runs":
        axes = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        while any(left):
            for a, n in enumerate(left):
                if n:
                    axes.append(a)
                    left[a] -= 1
    return torch.tensor(axes, dtype=torch.int32).to(device)


def rotary_axes(q, freqs, axes, positions, k=None, layout: str = "half", inverse: bool = False, scale: float = 1.0,
                out=None, k_out=None):
    """Rotary positions with several axes (time, height and width of images and video): as rotary(), but pair j turns by
    the position of axis ``axes[j]``. Returns the turned q, or (q, k).

    ``axes``: int32 of freqs' length (rotary_sections()); a pair whose axis is not one of positions' becomes NaN.
    ``positions``: int32 [axes, *q's leading shape], up to 16 axes. The others as in rotary().
    """
    lib = _lib.load()
    dev = _cuda(q)
    if layout not in _lib.ROTARY_LAYOUTS:
        raise ValueError("layout must be one of %s" % sorted(_lib.ROTARY_LAYOUTS))
    if q.dim() < 3:
        raise ValueError("q has shape %s, expected [..., heads, channels]" % (tuple(q.shape),))
    lead, (Hq, D), dt = q.shape[:-2], q.shape[-2:], q.dtype
    io = _io_code(dt)
    _need(q, "q", q.shape, dt, dev)
    _need(freqs, "freqs", (freqs.numel(),), torch.float64, dev)
    _need(axes, "axes", freqs.shape, torch.int32, dev)
    A = positions.shape[0] if positions.dim() else 0
    _need(positions, "positions", (A,) + lead, torch.int32, dev)
    Hk = 0
    if k is not None:
        Hk = k.shape[-2] if k.dim() == q.dim() else -1
        _need(k, "k", lead + (Hk, D), dt, dev)
        k_out = _result(k_out, "k_out", k)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if ((Hq + Hk) * D + freqs.numel()) >> 30 or A >> 31:
        _int32(A, Hq, Hk, D, 2 * freqs.numel())
    out = _result(out, "out", q)
    _call(dev, lib.kda_rotary_axes, _ptr(q), _ptr(k), _ptr(freqs), _ptr(axes), _ptr(positions), _ptr(out), _ptr(k_out),
          math.prod(lead), A, Hq, Hk, D, 2 * freqs.numel(), io, _lib.ROTARY_LAYOUTS[layout], int(bool(inverse)), scale)
    return out if k is None else (out, k_out)


# ---------------------------------------------------------------- layer norm
def _norm_args(x, weight, bias, o_gate):
    """(rows, groups, C) of x, with its parameters checked: weight and bias are [C], or [H, C] for x [..., H, C]."""
    dev = _cuda(x)
    if x.dim() < 1:
        raise ValueError("x has no channels")
    _need(x, "x", x.shape, x.dtype, dev)
    C, groups = x.shape[-1], 1
    p = weight if weight is not None else bias
    if p is not None:
        if p.dim() == 2 and x.dim() >= 2:
            groups = x.shape[-2]
        shape = (groups, C) if p.dim() == 2 else (C,)
        for name, t in (("weight", weight), ("bias", bias)):
            if t is not None:
                _need(t, name, shape, torch.float32, dev)
    if o_gate is not None:
        _need(o_gate, "o_gate", x.shape, x.dtype, dev)
    if groups * C >> 31:
        _int32(groups, C)
    return math.prod(x.shape[:-1]), max(groups, 1), C


def layer_norm_fwd(x, weight=None, bias=None, o_gate=None, eps: float = 1e-5, center: bool = True, out=None):
    """Layer norm over the last axis of x (bf16 or fp32, up to 16384 channels), then the optional output gate:
    ((x - mean) / sqrt(var + eps) * weight + bias) * sigmoid(o_gate).

    ``weight`` and ``bias``: fp32 [C], or [H, C] for x [..., H, C] (each head its own), or None. ``o_gate``: x's shape
    and dtype. ``center=False`` leaves the mean in (and takes the mean square for the variance).
    """
    lib = _lib.load()
    io = _io_code(x.dtype)
    rows, groups, C = _norm_args(x, weight, bias, o_gate)
    dev = x.device
    out = _result(out, "out", x)
    _call(dev, lib.kda_layer_norm_fwd, _ptr(x), _ptr(weight), _ptr(bias), _ptr(o_gate), _ptr(out), rows, groups, C, eps,
          int(bool(center)), io)
    return out


def layer_norm_bwd(dy, x, weight=None, bias=None, o_gate=None, eps: float = 1e-5, center: bool = True, workspace=None,
                   out=None):
    """Gradients of layer_norm_fwd given ``dy`` (x's shape and dtype) and its arguments. Returns a dict: dx;
    dweight and dbias (fp32) for the parameters given; do_gate with ``o_gate``. ``out`` may hold preallocated results
    by these names. Deterministic. ``x`` may be a Checkpoint8: the gradients are those at the values it stands for, and
    the kernel reads its codes."""
    lib = _lib.load()
    saved = x if isinstance(x, Checkpoint8) else None
    if saved is not None:
        x = dy  # of the shape and dtype that the checkpoint has to have
        if saved.dtype is not dy.dtype:
            raise TypeError("x stands for %s, dy has dtype %s" % (saved.dtype, dy.dtype))
        _need8(saved, "x", dy.shape, _cuda(dy))
    io = _io_code(x.dtype)
    rows, groups, C = _norm_args(x, weight, bias, o_gate)
    dev, dt = x.device, x.dtype
    _need(dy, "dy", x.shape, dt, dev)
    like = {"dx": x}
    if weight is not None:
        like["dweight"] = weight
    if bias is not None:
        like["dbias"] = bias
    if o_gate is not None:
        like["do_gate"] = o_gate
    given = out or {}
    for name in given:
        if name not in like:
            raise ValueError("out[%r]: not a result of this call" % (name,))
    workspace = _workspace(workspace, lib.kda_layer_norm_bwd_workspace_bytes(rows, groups, C), dev,
                           "layer_norm_bwd(rows=%d, groups=%d, C=%d)", rows, groups, C)
    res = {n: _result(given.get(n), n, t) for n, t in like.items()}
    if saved is None:
        fn, inputs = lib.kda_layer_norm_bwd, (_ptr(x),)
    else:
        fn, inputs = lib.kda_layer_norm_bwd_checkpoint8, (_ptr(saved.codes), _ptr(saved.scales))
    _call(dev, fn, _ptr(dy), *inputs, _ptr(weight), _ptr(bias), _ptr(o_gate), _ptr(res["dx"]),
          _ptr(res.get("dweight")), _ptr(res.get("dbias")), _ptr(res.get("do_gate")), rows, groups, C, eps,
          int(bool(center)), io, _ptr(workspace), workspace.numel())
    return res
