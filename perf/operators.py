"""The operators around the recurrence, as they are measured: linear attention with one decay per head (chunked
forward, backward, single-token step), rotary positions, and layer norm with its gradient.

``run`` makes the package's calls where ``own`` is true; elsewhere it computes the same in elementary torch
operations, in fp32 (decay sums and rotary angles in fp64), rounded once at the end. ``exact`` is the definition in
fp64: the linear attention as the masked quadratic form over whole sequences, one head at a time.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64  # tokens per block of the plain chunk form


def listed():
    return [
        # a short prompt of a tiny layer: what a call costs at the least
        dict(name="hd_fwd_tiny", op="hd_fwd", io="fp32", B=1, T=64, seqs=0, H=2, Hk=2, K=32, V=32, decay="token",
             S0=False),
        # one 4096-token sequence of 96 heads of 128 channels: the benchmark's prefill shape
        dict(name="hd_fwd_4k", op="hd_fwd", io="bf16", B=1, T=4096, seqs=0, H=96, Hk=96, K=128, V=128, decay="token",
             S0=False),
        # sixteen packed prompts of ragged lengths that continue from states, shared q/k heads, fixed decays
        dict(name="hd_fwd_packed", op="hd_fwd", io="bf16", B=1, T=17011, seqs=16, H=32, Hk=8, K=128, V=64,
             decay="head", S0=True),
        # a training step's gradients at the benchmark's shape
        dict(name="hd_bwd_4k", op="hd_bwd", io="bf16", B=1, T=4096, seqs=0, H=96, Hk=96, K=128, V=128, decay="token",
             S0=False),
        # gradients of a packed batch of odd lengths in fp32, through states and their gradients
        dict(name="hd_bwd_packed", op="hd_bwd", io="fp32", B=1, T=1531, seqs=5, H=12, Hk=4, K=64, V=128,
             decay="token", S0=True),
        # one token of one stream, and of 512 streams (3.2 GB of states)
        dict(name="hd_decode_1", op="hd_decode", io="bf16", N=1, H=96, Hk=96, K=128, V=128, decay="token"),
        dict(name="hd_decode_512", op="hd_decode", io="bf16", N=512, H=96, Hk=96, K=128, V=128, decay="head"),
        # the new tokens' q and k of 32 streams far into their contexts; a whole prompt's, rotated in part of the
        # head and backwards, as its gradient is
        dict(name="rotary_decode", op="rotary", io="bf16", B=0, T=32, H=32, Hk=8, D=128, R=128, layout="half",
             inverse=False, far=True),
        dict(name="rotary_prompt", op="rotary", io="bf16", B=2, T=8191, H=32, Hk=32, D=128, R=64,
             layout="interleaved", inverse=True, far=False),
        # the recurrence's output normed head by head and gated; rows of the model's width and their gradients, and
        # an odd width in fp32
        dict(name="norm_heads", op="norm_fwd", io="bf16", rows=4096, G=96, C=128, gate=True, center=False),
        dict(name="norm_bwd_wide", op="norm_bwd", io="bf16", rows=8192, G=1, C=4096, gate=False, center=True),
        dict(name="norm_bwd_odd", op="norm_bwd", io="fp32", rows=1003, G=3, C=333, gate=True, center=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["hd_fwd", "hd_fwd", "hd_bwd", "hd_bwd", "hd_decode", "rotary", "norm_fwd", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("hd_fwd", "hd_bwd"):
        K, V = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        Hk = _spread(rng, 1, 24)
        H = Hk * rng.choice([1, 1, 2, 4])
        T = _spread(rng, 1, min(8192, (4096 * 96) // H))
        seqs = rng.choice([0, 0, 1, 3, 8])
        B = 1 if seqs else rng.choice([1, 1, 2])
        return dict(op=op, io=io, B=B, T=max(T // B, seqs, 1), seqs=seqs, H=H, Hk=Hk, K=K, V=V,
                    decay=rng.choice(["token", "token", "head"]), S0=rng.random() < 0.5)
    if op == "hd_decode":
        Hk = _spread(rng, 1, 48)
        return dict(op=op, io=io, N=_spread(rng, 1, 512), H=Hk * rng.choice([1, 2]), Hk=Hk,
                    K=rng.choice([32, 64, 128]), V=rng.choice([32, 64, 128]), decay=rng.choice(["token", "head"]))
    if op == "rotary":
        Hk = _spread(rng, 1, 16)
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        return dict(op=op, io=io, B=rng.choice([0, 1, 2]), T=_spread(rng, 1, 6000), H=Hk * rng.choice([1, 2, 4]),
                    Hk=Hk, D=D, R=rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5, far=rng.random() < 0.5)
    G = rng.choice([1, 1, _spread(rng, 1, 64)])
    C = _spread(rng, 16, 9000) if G == 1 else rng.choice([32, 64, 100, 128])
    return dict(op=op, io=io, rows=_spread(rng, 1, max(1, min(20000, (8192 * 4096) // (G * C)))), G=G, C=C,
                gate=rng.random() < 0.5, center=rng.random() < 0.7)


# ------------------------------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """The sequences' lengths: ragged, summing to T, some of them possibly empty where there is little to share."""
    if not case["seqs"]:
        return [case["T"]] * case["B"]
    cuts = np.sort(np.random.default_rng([seed, 77]).integers(0, case["T"] + 1, case["seqs"] - 1))
    return np.diff(np.concatenate([[0], cuts, [case["T"]]])).tolist()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["io"]]

    def randn(*shape, dtype=dt, std=1.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).to(dtype)

    def decay(*shape):
        # log-decays of about -0.05 a step (windows of some tens of tokens), spread over two decades
        return -torch.exp(torch.randn(shape, generator=gen, device=dev) - 3.0)

    st = dict(case=dict(case), op=case["op"])
    if case["op"] in ("hd_fwd", "hd_bwd"):
        B, T, H, Hk, K, V = (case[n] for n in ("B", "T", "H", "Hk", "K", "V"))
        lengths = _lengths(case, seed)
        N = len(lengths)
        st.update(q=randn(B, T, Hk, K), k=randn(B, T, Hk, K, std=K ** -0.5), v=randn(B, T, H, V),
                  g=decay(B, T, H).to(dt) if case["decay"] == "token" else decay(H),
                  S0=randn(N, H, K, V, dtype=torch.float32, std=0.02) if case["S0"] else None,
                  scale=K ** -0.5, lengths=lengths, cu=None)
        if case["seqs"]:
            st["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        if case["op"] == "hd_bwd":
            st["do"] = randn(B, T, H, V)
            st["dS"] = randn(N, H, K, V, dtype=torch.float32, std=0.02) if case["S0"] else None
    elif case["op"] == "hd_decode":
        N, H, Hk, K, V = (case[n] for n in ("N", "H", "Hk", "K", "V"))
        st.update(q=randn(N, Hk, K), k=randn(N, Hk, K, std=K ** -0.5), v=randn(N, H, V),
                  g=decay(N, H).to(dt) if case["decay"] == "token" else decay(H), scale=K ** -0.5,
                  S=randn(N, H, K, V, dtype=torch.float32, std=0.5))
    elif case["op"] == "rotary":
        lead = (case["B"], case["T"]) if case["B"] else (case["T"],)
        st.update(q=randn(*lead, case["H"], case["D"]), k=randn(*lead, case["Hk"], case["D"]))
        R = case["R"]
        st["freqs"] = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
        st["pos"] = None
        if case["far"] or not case["B"]:
            st["pos"] = torch.randint(0, (1 << 20) if case["far"] else 4096, lead, generator=gen, device=dev,
                                      dtype=torch.int32)
    else:
        rows, G, C = case["rows"], case["G"], case["C"]
        shape = (rows, G, C) if G > 1 else (rows, C)
        wshape = (G, C) if G > 1 else (C,)
        st.update(x=randn(*shape) + (0.5 if case["center"] else 0.0), w=1.0 + randn(*wshape, dtype=torch.float32, std=0.2),
                  b=randn(*wshape, dtype=torch.float32, std=0.2) if case["center"] else None,
                  z=randn(*shape) if case["gate"] else None)
        if case["op"] == "norm_bwd":
            st["dy"] = randn(*shape)
    return st


# ------------------------------------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return {"hd_fwd": _hd_fwd, "hd_bwd": _hd_bwd, "hd_decode": _hd_decode, "rotary": _rotary, "norm_fwd": _norm_fwd,
            "norm_bwd": _norm_bwd}[state["op"]](state)


def _run_own(s):
    import kda_gated_delta_chunk_amd as kda

    c = s["case"]
    if s["op"] == "hd_fwd":
        o, S = kda.hd_chunk_fwd(s["q"], s["k"], s["v"], s["g"], S0=s["S0"], cu_seqlens=s["cu"], scale=s["scale"])
        return {"o": o, "S": S}
    if s["op"] == "hd_bwd":
        return kda.hd_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], S0=s["S0"], dS_final=s["dS"],
                                cu_seqlens=s["cu"], scale=s["scale"])
    if s["op"] == "hd_decode":
        o = kda.hd_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], scale=s["scale"])
        return {"o": o, "S": s["S"]}
    if s["op"] == "rotary":
        q, k = kda.rotary(s["q"], s["freqs"], k=s["k"], positions=s["pos"], layout=c["layout"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if s["op"] == "norm_fwd":
        return {"y": kda.layer_norm_fwd(s["x"], weight=s["w"], bias=s["b"], o_gate=s["z"], center=c["center"])}
    return kda.layer_norm_bwd(s["dy"], s["x"], weight=s["w"], bias=s["b"], o_gate=s["z"], center=c["center"])


def _blocks(s):
    """Token indexes [blocks, CHUNK] of every sequence cut into blocks, which of them are tokens, each block's
    sequence, and per block the first block of its sequence."""
    dev = s["q"].device
    n = torch.tensor(s["lengths"], device=dev)
    nb = (n + CHUNK - 1) // CHUNK
    total = sum((x + CHUNK - 1) // CHUNK for x in s["lengths"])
    seq = torch.repeat_interleave(torch.arange(len(s["lengths"]), device=dev), nb, output_size=total)
    first = (torch.cumsum(nb, 0) - nb)[seq]
    start = torch.cumsum(n, 0) - n
    at = (torch.arange(total, device=dev) - first)[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    valid = at < n[seq][:, None]
    idx = torch.where(valid, start[seq][:, None] + at, 0)
    return idx, valid, seq, first


def _cut(x, idx, valid, H):
    """[B, T, heads, D] as fp32 blocks [H, blocks, CHUNK, D], heads repeated to H, zeros where no token is."""
    x = x.reshape(-1, x.shape[-2], x.shape[-1])[idx].float() * valid[:, :, None, None]
    return x.repeat_interleave(H // x.shape[2], dim=2).permute(2, 0, 1, 3).contiguous()


def _join(x, idx, valid, like, heads):
    """Blocks [H, blocks, CHUNK, D] back to [B, T, heads, D], summed over the v heads that share a q/k head."""
    H, nb, C, D = x.shape
    x = x.reshape(heads, H // heads, nb, C, D).sum(1).permute(1, 2, 0, 3)
    out = torch.zeros(like.shape[0] * like.shape[1], heads, D, dtype=x.dtype, device=x.device)
    out[idx[valid]] = x[valid]
    return out.reshape(like.shape[0], like.shape[1], heads, D).to(like.dtype)


def _decays(s, idx, valid, seq):
    """Sums of the log-decays in fp64: inside the blocks [H, blocks, CHUNK] and over whole blocks [H, blocks]."""
    H = s["v"].shape[2]
    g = s["g"].double()
    g = g.reshape(-1, H)[idx] if g.dim() == 3 else g.expand(idx.shape[0], CHUNK, H)
    b = torch.cumsum(g * valid[:, :, None], 1).permute(2, 0, 1)
    return b, torch.cumsum(b[:, :, -1], 1)


def _states(s, inc, Bc, seq, first):
    """States at the blocks' starts [H, blocks, K, V] and at the sequences' ends [H, sequences, K, V]."""
    H, nb, K, V = inc.shape
    at = torch.arange(nb, device=inc.device)
    Bprev = torch.cat([torch.zeros_like(Bc[:, :1]), Bc[:, :-1]], 1)
    M = torch.where((at[:, None] > at) & (seq[:, None] == seq), torch.exp(Bprev[:, :, None] - Bc[:, None, :]), 0.0)
    S = (M.float() @ inc.reshape(H, nb, K * V)).reshape(H, nb, K, V)
    N = len(s["lengths"])
    mine = seq == torch.arange(N, device=inc.device)[:, None]
    last = torch.where(mine, at, -1).amax(1).clamp(min=0) if nb else None
    F = torch.where(mine, torch.exp(Bc[:, last][:, :, None] - Bc[:, None, :]), 0.0)
    Sf = (F.float() @ inc.reshape(H, nb, K * V)).reshape(H, N, K, V)
    if s["S0"] is not None:
        S0 = s["S0"].permute(1, 0, 2, 3)
        S = S + torch.exp(Bprev - Bprev[:, first]).float()[..., None, None] * S0[:, seq]
        tot = torch.where(mine, (Bc - Bprev)[:, None, :], 0.0).sum(-1)
        Sf = Sf + torch.exp(tot).float()[..., None, None] * S0
    return S, Sf


def _mask(b):
    """exp(b_i - b_j) for j <= i, else 0."""
    i = torch.arange(CHUNK, device=b.device)
    d = torch.where(i[:, None] >= i, b[..., :, None] - b[..., None, :], -math.inf)
    return torch.exp(d.float())


def _hd_fwd(s):
    idx, valid, seq, first = _blocks(s)
    H = s["v"].shape[2]
    q, k, v = (_cut(s[n], idx, valid, H) for n in ("q", "k", "v"))
    b, Bc = _decays(s, idx, valid, seq)
    w = torch.exp(b[:, :, -1:] - b).float()[..., None]
    S, Sf = _states(s, (k * w).transpose(2, 3) @ v, Bc, seq, first)
    o = ((q @ k.transpose(2, 3)) * _mask(b)) @ v + torch.exp(b).float()[..., None] * (q @ S)
    return {"o": _join(s["scale"] * o, idx, valid, s["v"], H), "S": Sf.permute(1, 0, 2, 3).contiguous()}


def _hd_bwd(s):
    idx, valid, seq, first = _blocks(s)
    H, Hk = s["v"].shape[2], s["q"].shape[2]
    q, k, v, do = (_cut(s[n], idx, valid, H) for n in ("q", "k", "v", "do"))
    do = s["scale"] * do
    b, Bc = _decays(s, idx, valid, seq)
    eb, w = torch.exp(b).float()[..., None], torch.exp(b[:, :, -1:] - b).float()[..., None]
    inc, dinc = (k * w).transpose(2, 3) @ v, (q * eb).transpose(2, 3) @ do
    S, Sf = _states(s, inc, Bc, seq, first)
    # state gradients at the blocks' ends and at the sequences' starts
    nb, K, V = inc.shape[1], inc.shape[2], inc.shape[3]
    at = torch.arange(nb, device=inc.device)
    Bprev = torch.cat([torch.zeros_like(Bc[:, :1]), Bc[:, :-1]], 1)
    M = torch.where((at > at[:, None]) & (seq[:, None] == seq), torch.exp(Bprev[:, None, :] - Bc[:, :, None]), 0.0)
    E = (M.float() @ dinc.reshape(H, nb, K * V)).reshape(H, nb, K, V)
    N = len(s["lengths"])
    mine = seq == torch.arange(N, device=inc.device)[:, None]
    F = torch.where(mine, torch.exp(Bprev - Bprev[:, first])[:, None, :], 0.0)
    dS0 = (F.float() @ dinc.reshape(H, nb, K * V)).reshape(H, N, K, V)
    if s["dS"] is not None:
        dS = s["dS"].permute(1, 0, 2, 3)
        last = torch.where(mine, at, -1).amax(1).clamp(min=0)
        E = E + torch.exp(Bc[:, last[seq]] - Bc).float()[..., None, None] * dS[:, seq]
        tot = torch.where(mine, (Bc - Bprev)[:, None, :], 0.0).sum(-1)
        dS0 = dS0 + torch.exp(tot).float()[..., None, None] * dS
    D = _mask(b)
    P, dP = (q @ k.transpose(2, 3)) * D, (do @ v.transpose(2, 3)) * D
    dq = dP @ k + eb * (do @ S.transpose(2, 3))
    dk = dP.transpose(2, 3) @ q + w * (v @ E.transpose(2, 3))
    dv = P.transpose(2, 3) @ do + w * (k @ E)
    out = {"dq": _join(dq, idx, valid, s["q"], Hk), "dk": _join(dk, idx, valid, s["k"], Hk),
           "dv": _join(dv, idx, valid, s["v"], H), "dS0": dS0.permute(1, 0, 2, 3).contiguous()}
    if s["g"].dim() == 3:
        # a token's log-decay acts on every pair and state that spans its border: rows' sums less columns' sums
        # after it in the block, and what the block's end passes on
        X = (q @ k.transpose(2, 3)) * dP
        r = X.sum(3) + (q * eb * (do @ S.transpose(2, 3))).sum(3)
        c = X.sum(2) + (v * w * (k @ E)).sum(3)
        end = torch.exp(b[:, :, -1]).float()[..., None, None] * S + inc
        after = torch.flip(torch.cumsum(torch.flip((r - c).double(), [2]), 2), [2])
        dg = after + (end * E).double().sum((2, 3))[..., None]
        out["dg"] = _join(dg[..., None], idx, valid, s["g"][..., None], H)[..., 0]
    return out


def _hd_decode(s):
    H, G = s["v"].shape[1], s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(G, dim=1) for n in ("q", "k"))
    a = torch.exp(s["g"].float()).expand(s["v"].shape[0], H)
    s["S"].mul_(a[..., None, None]).add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = (s["scale"] * (q[..., None, :] @ s["S"]))[..., 0, :]
    return {"o": o.to(s["v"].dtype), "S": s["S"]}


def _turn(x, cos, sin, layout):
    R = 2 * cos.shape[-1]
    y = x.float()
    a, b = (y[..., :R // 2], y[..., R // 2:R]) if layout == "half" else (y[..., 0:R:2], y[..., 1:R:2])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([r, y[..., R:]], -1).to(x.dtype)


def _rotary(s):
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["T"], device=s["q"].device)
    angle = pos.double()[..., None, None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float() * (-1.0 if c["inverse"] else 1.0)
    return {"q": _turn(s["q"], cos, sin, c["layout"]), "k": _turn(s["k"], cos, sin, c["layout"])}


EPS = 1e-5


def _normed(s):
    x = s["x"].float()
    if s["case"]["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_fwd(s):
    y = _normed(s)[0] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    if s["z"] is not None:
        y = y * torch.sigmoid(s["z"].float())
    return {"y": y.to(s["x"].dtype)}


def _norm_bwd(s):
    n, r = _normed(s)
    dy, out = s["dy"].float(), {}
    if s["z"] is not None:
        a = torch.sigmoid(s["z"].float())
        y = n * s["w"] + (s["b"] if s["b"] is not None else 0.0)
        out["do_gate"] = (dy * y * a * (1.0 - a)).to(s["x"].dtype)
        dy = dy * a
    out["dweight"] = (dy * n).sum(0)
    if s["b"] is not None:
        out["dbias"] = dy.sum(0)
    d = dy * s["w"]
    dx = d - n * (d * n).mean(-1, keepdim=True)
    if s["case"]["center"]:
        dx = dx - d.mean(-1, keepdim=True)
    out["dx"] = (r * dx).to(s["x"].dtype)
    return out


# ------------------------------------------------------------------------------------------------- work
def _size(shape, io):
    return math.prod(shape) * (2 if io == "bf16" else 4)


def work(case):
    io = case["io"]
    e = 2 if io == "bf16" else 4
    if case["op"] in ("hd_fwd", "hd_bwd"):
        B, T, H, Hk, K, V = (case[n] for n in ("B", "T", "H", "Hk", "K", "V"))
        states = (case["seqs"] or B) * H * K * V * 4
        qk, v = 2 * B * T * Hk * K * e, B * T * H * V * e
        g = B * T * H * e if case["decay"] == "token" else 4 * H
        if case["op"] == "hd_fwd":
            return {"bytes": qk + 2 * v + g + states * (2 if case["S0"] else 1), "flops": 4 * B * T * H * K * V}
        dg = g if case["decay"] == "token" else 0
        return {"bytes": 2 * qk + 3 * v + g + dg + states * (3 if case["S0"] else 1), "flops": 10 * B * T * H * K * V}
    if case["op"] == "hd_decode":
        N, H, Hk, K, V = (case[n] for n in ("N", "H", "Hk", "K", "V"))
        g = N * H * e if case["decay"] == "token" else 4 * H
        return {"bytes": 8 * N * H * K * V + e * (2 * N * Hk * K + 2 * N * H * V) + g, "flops": 5 * N * H * K * V}
    if case["op"] == "rotary":
        n = max(case["B"], 1) * case["T"]
        x = n * (case["H"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * e * x + (4 * n if case["far"] or not case["B"] else 0) + 4 * case["R"],
                "flops": 3 * n * (case["H"] + case["Hk"]) * case["R"]}
    x, w = case["rows"] * case["G"] * case["C"], case["G"] * case["C"] * 4
    params = 2 if case["center"] else 1
    if case["op"] == "norm_fwd":
        return {"bytes": e * x * (3 if case["gate"] else 2) + params * w, "flops": 8 * x}
    return {"bytes": e * x * (5 if case["gate"] else 3) + 2 * params * w, "flops": 16 * x}


# ------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    def quadratic(s, bwd):
        """The masked quadratic form, one sequence and v head at a time."""
        dev, f64 = s["q"].device, torch.float64
        B, T, H, V = s["v"].shape
        Hk, K = s["q"].shape[2:]
        N = len(s["lengths"])
        flat = {n: s[n].reshape(B * T, s[n].shape[2], s[n].shape[3]) for n in ("q", "k", "v", "do") if n in s}
        o = torch.zeros(B * T, H, V, dtype=f64, device=dev)
        Sf = torch.zeros(N, H, K, V, dtype=f64, device=dev)
        dq, dk = (torch.zeros(B * T, Hk, K, dtype=f64, device=dev) for _ in range(2))
        dv, dg = torch.zeros_like(o), torch.zeros(B * T, H, dtype=f64, device=dev)
        dS0 = torch.zeros_like(Sf)
        begin = 0
        for n, L in enumerate(s["lengths"]):
            t = slice(begin, begin + L)
            begin += L
            for h in range(H):
                hk = h * Hk // H
                S0 = s["S0"][n, h].double() if s["S0"] is not None else torch.zeros(K, V, dtype=f64, device=dev)
                dS = s["dS"][n, h].double() if bwd and s["dS"] is not None else torch.zeros(K, V, dtype=f64, device=dev)
                if L == 0:
                    Sf[n, h], dS0[n, h] = S0, dS
                    continue
                g = s["g"].reshape(B * T, H)[t, h].double() if s["g"].dim() == 3 else s["g"][h].double().expand(L)
                q, k, v = flat["q"][t, hk].double(), flat["k"][t, hk].double(), flat["v"][t, h].double()
                b = torch.cumsum(g, 0)
                D = torch.exp(torch.tril(b[:, None] - b)).tril()
                A = (q @ k.T) * D
                enter, leave = torch.exp(b)[:, None], torch.exp(b[-1] - b)[:, None]
                Sf[n, h] = (k * leave).T @ v + torch.exp(b[-1]) * S0
                o[t, h] = s["scale"] * (A @ v + enter * (q @ S0))
                if not bwd:
                    continue
                do = s["scale"] * flat["do"][t, h].double()
                dA = do @ v.T
                dq[t, hk] += (dA * D) @ k + enter * (do @ S0.T)
                dk[t, hk] += (dA * D).T @ q + leave * (v @ dS.T)
                dv[t, h] = A.T @ do + leave * (k @ dS)
                dS0[n, h] = (q * enter).T @ do + torch.exp(b[-1]) * dS
                # dL/db: every weight is exp of a difference of b's
                X = A * dA
                db = X.sum(1) - X.sum(0) + (enter * q * (do @ S0.T)).sum(1) - (leave * v * (k @ dS)).sum(1)
                db[-1] += (Sf[n, h] * dS).sum()
                dg[t, h] = torch.flip(torch.cumsum(torch.flip(db, [0]), 0), [0])
        if not bwd:
            return {"o": o.reshape(B, T, H, V), "S": Sf}
        out = {"dq": dq.reshape(B, T, Hk, K), "dk": dk.reshape(B, T, Hk, K), "dv": dv.reshape(B, T, H, V), "dS0": dS0}
        if s["g"].dim() == 3:
            out["dg"] = dg.reshape(B, T, H)
        return out

    s = prepare(case, seed)
    if case["op"] in ("hd_fwd", "hd_bwd"):
        if sum(n * n for n in s["lengths"]) * case["H"] * case["K"] > 2e12:
            return None
        return quadratic(s, case["op"] == "hd_bwd")
    if case["op"] == "hd_decode":
        N, H, K, V = s["S"].shape
        out, G = torch.empty(N, H, V, dtype=torch.float64, device=s["S"].device), H // s["q"].shape[1]
        Sn = torch.empty(N, H, K, V, dtype=torch.float64, device=s["S"].device)
        a = s["g"].double().exp().expand(N, H)
        for h in range(H):
            Sn[:, h] = a[:, h, None, None] * s["S"][:, h] + torch.einsum("nk,nv->nkv", s["k"][:, h // G].double(),
                                                                        s["v"][:, h].double())
            out[:, h] = s["scale"] * (s["q"][:, h // G, :, None].double() * Sn[:, h]).sum(1)
        return {"o": out, "S": Sn}
    if case["op"] == "rotary":
        pos = s["pos"].cpu().numpy() if s["pos"] is not None else np.arange(case["T"])
        # e^{i angle} in complex numbers
        turn = np.exp((-1j if case["inverse"] else 1j) * (pos.astype(np.float64)[..., None] * s["freqs"].cpu().numpy()))
        turn = torch.from_numpy(turn).to(s["q"].device)[..., None, :]
        out = {}
        for n in ("q", "k"):
            x = s[n].double()
            y = x.clone()
            R = case["R"]
            even, odd = (slice(0, R // 2), slice(R // 2, R)) if case["layout"] == "half" else (slice(0, R, 2),
                                                                                              slice(1, R, 2))
            z = torch.complex(x[..., even], x[..., odd]) * turn
            y[..., even], y[..., odd] = z.real, z.imag
            out[n] = y
        return out
    x = s["x"].double()
    mu = x.mean(-1, keepdim=True) if case["center"] else 0.0
    sd = torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + EPS)
    w = s["w"].double()
    b = s["b"].double() if s["b"] is not None else 0.0
    a = 1.0 / (1.0 + torch.exp(-s["z"].double())) if s["z"] is not None else 1.0
    if case["op"] == "norm_fwd":
        return {"y": ((x - mu) / sd * w + b) * a}
    dy, C = s["dy"].double(), x.shape[-1]
    out = {}
    if s["z"] is not None:
        out["do_gate"] = dy * ((x - mu) / sd * w + b) * a * (1.0 - a)
    dn = dy * a * w
    # through the standard deviation and the mean, one after the other
    dsd = -(dn * (x - mu)).sum(-1, keepdim=True) / sd ** 2
    dc = dn / sd + dsd * (x - mu) / (C * sd)
    out["dx"] = dc - dc.sum(-1, keepdim=True) / C if case["center"] else dc
    out["dweight"] = (dy * a * (x - mu) / sd).sum(0)
    if s["b"] is not None:
        out["dbias"] = (dy * a).sum(0)
    return out
