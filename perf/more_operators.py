"""More operators around the recurrence, as they are measured: the gated delta rule with one decay per head (chunked
forward, backward, single-token step), rotary positions with several axes, and activation checkpoints in 8 bits with
the backward passes that read them.

``run`` makes the package's calls where ``own`` is true; elsewhere it computes the same in elementary torch
operations, in fp32 (decay sums, rotary angles and long sums in fp64), rounded once at the end. ``exact`` is the
definition in fp64: the gated delta rule token by token.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 32  # tokens per block of the plain chunk form
BLOCK = 128  # values that share a scale in a checkpoint
EPS = 1e-5


def listed():
    return [
        # a short prompt of a tiny layer: what a call costs at the least
        dict(name="gd_fwd_tiny", op="gd_fwd", io="fp32", gates="fp32", B=1, T=64, seqs=0, H=2, Hk=2, K=32, V=32,
             S0=False),
        # one 4096-token sequence of 96 heads of 128 channels: the benchmark's prefill shape
        dict(name="gd_fwd_4k", op="gd_fwd", io="bf16", gates="bf16", B=1, T=4096, seqs=0, H=96, Hk=96, K=128, V=128,
             S0=False),
        # sixteen packed prompts of ragged lengths that continue from states, two v heads for each q/k head
        dict(name="gd_fwd_packed", op="gd_fwd", io="bf16", gates="fp32", B=1, T=17011, seqs=16, H=32, Hk=16, K=128,
             V=128, S0=True),
        # a training step's gradients at the benchmark's shape
        dict(name="gd_bwd_4k", op="gd_bwd", io="bf16", gates="bf16", B=1, T=4096, seqs=0, H=96, Hk=96, K=128, V=128,
             S0=False),
        # gradients of a packed batch of odd lengths in fp32, through states and their gradients
        dict(name="gd_bwd_packed", op="gd_bwd", io="fp32", gates="fp32", B=1, T=1531, seqs=5, H=12, Hk=4, K=64, V=128,
             S0=True),
        # the gradients of a layer whose q, k and v were kept in 8 bits
        dict(name="gd_bwd8_2k", op="gd_bwd8", io="bf16", gates="fp32", B=2, T=2050, seqs=0, H=32, Hk=16, K=128, V=128,
             S0=False),
        # one token of 512 streams (3.2 GB of states)
        dict(name="gd_decode_512", op="gd_decode", io="bf16", gates="bf16", N=512, H=96, Hk=96, K=128, V=128),
        # the new tokens' q and k of 32 streams, and a batch of two clips: three axes, their pairs in runs and in turns
        dict(name="axes_decode", op="axes", io="bf16", B=0, T=32, H=32, Hk=8, D=128, sections="16 24 24",
             order="runs", layout="half", inverse=False, far=True),
        dict(name="axes_clips", op="axes", io="bf16", B=2, T=8191, H=32, Hk=8, D=128, sections="24 20 20",
             order="turns", layout="half", inverse=False, far=False),
        # a block's input of the model's width into a checkpoint and back out of it
        dict(name="ckpt_wide", op="ckpt", io="bf16", rows=8192, G=1, C=4096),
        # a norm's gradients from the checkpoint of its input, and an odd width in fp32
        dict(name="norm_bwd8_wide", op="norm_bwd8", io="bf16", rows=8192, G=1, C=4096, gate=False, center=False),
        dict(name="norm_bwd8_odd", op="norm_bwd8", io="fp32", rows=1003, G=3, C=333, gate=True, center=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gd_fwd", "gd_fwd", "gd_fwd", "gd_bwd", "gd_bwd", "gd_bwd8", "gd_decode", "axes", "axes", "ckpt",
                     "norm_bwd8"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    gates = rng.choice([io, "fp32"])
    if op in ("gd_fwd", "gd_bwd", "gd_bwd8"):
        K, V = rng.choice([32, 64, 128]), rng.choice([32, 64, 128, 128])
        Hk = _spread(rng, 1, 24)
        H = Hk * rng.choice([1, 1, 2, 4])
        T = _spread(rng, 1, min(8192, (4096 * 96) // H))
        seqs = rng.choice([0, 0, 1, 3, 8])
        B = 1 if seqs else rng.choice([1, 1, 2])
        return dict(op=op, io=io, gates=gates, B=B, T=max(T // B, 1), seqs=seqs, H=H, Hk=Hk, K=K, V=V,
                    S0=rng.random() < 0.5)
    if op == "gd_decode":
        Hk = _spread(rng, 1, 48)
        return dict(op=op, io=io, gates=gates, N=_spread(rng, 1, 512), H=Hk * rng.choice([1, 2]), Hk=Hk,
                    K=rng.choice([32, 64, 128]), V=rng.choice([32, 64, 128]))
    if op == "axes":
        Hk = _spread(rng, 1, 16)
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        axes = rng.choice([2, 3, 3])
        pairs = rng.choice([D // 2, D // 2, D // 4, rng.randint(axes, D // 2)])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        return dict(op=op, io=io, B=rng.choice([0, 1, 2]), T=_spread(rng, 1, 6000), H=Hk * rng.choice([1, 2, 4]),
                    Hk=Hk, D=D, sections=sections, order=rng.choice(["runs", "turns"]),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5, far=rng.random() < 0.5)
    G = rng.choice([1, 1, _spread(rng, 1, 64)])
    C = _spread(rng, 16, 9000) if G == 1 else rng.choice([32, 64, 100, 128])
    rows = _spread(rng, 1, max(1, min(20000, (8192 * 4096) // (G * C))))
    if op == "ckpt":
        return dict(op=op, io=io, rows=rows, G=G, C=C)
    return dict(op=op, io=io, rows=rows, G=G, C=C, gate=rng.random() < 0.5, center=rng.random() < 0.7)


# ------------------------------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """The sequences' lengths: ragged, summing to T, some of them possibly empty where there is little to share."""
    if not case["seqs"]:
        return [case["T"]] * case["B"]
    cuts = np.sort(np.random.default_rng([seed, 78]).integers(0, case["T"] + 1, case["seqs"] - 1))
    return np.diff(np.concatenate([[0], cuts, [case["T"]]])).tolist()


def _sections(case):
    """How many channel pairs each axis turns."""
    return [int(n) for n in case["sections"].split()]


def _pair_axes(sections, order):
    """The axis of every channel pair: the sections one after the other, or the axes in turns while they last."""
    if order == "runs":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _to_blocks(x):
    C = x.shape[-1]
    nb = (C + BLOCK - 1) // BLOCK
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - C))
    return x.reshape(*x.shape[:-1], nb, BLOCK)


def _save8(x):
    """Codes (whole numbers of at most 127 in size) and each block's step: its largest value's 127th part."""
    b = _to_blocks(x.float())
    top = b.abs().amax(-1)
    codes = torch.where(top[..., None] > 0, torch.round(b * 127.0 / top[..., None]), 0.0)
    return codes.flatten(-2)[..., :x.shape[-1]].to(torch.int8), top / 127.0


def _restore8(codes, scales, dtype):
    return (_to_blocks(codes.float()) * scales[..., None]).flatten(-2)[..., :codes.shape[-1]].to(dtype)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["io"]]

    def randn(*shape, dtype=dt, std=1.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).to(dtype)

    def unit(*shape):  # rows of length one, as the recurrence's keys and queries are
        x = torch.randn(shape, generator=gen, device=dev)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    st = dict(case=dict(case), op=case["op"])
    if case["op"].startswith("gd"):
        H, Hk, K, V = (case[n] for n in ("H", "Hk", "K", "V"))
        gt = DTYPES[case["gates"]]
        decode = case["op"] == "gd_decode"
        lead = (case["N"],) if decode else (case["B"], case["T"])
        # log-decays of about -0.05 a step (windows of some tens of tokens), spread over two decades; write strengths
        # over (0, 1)
        st.update(q=unit(*lead, Hk, K), k=unit(*lead, Hk, K), v=randn(*lead, H, V),
                  g=(-torch.exp(torch.randn((*lead, H), generator=gen, device=dev) - 3.0)).to(gt),
                  beta=torch.sigmoid(torch.randn((*lead, H), generator=gen, device=dev)).to(gt), scale=K ** -0.5)
        if decode:
            st["S"] = randn(case["N"], H, K, V, dtype=torch.float32, std=0.5)
            return st
        lengths = _lengths(case, seed)
        N = len(lengths)
        st.update(lengths=lengths, cu=None,
                  S0=randn(N, H, K, V, dtype=torch.float32, std=0.1) if case["S0"] else None)
        if case["seqs"]:
            st["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        if case["op"] != "gd_fwd":
            st["do"] = randn(*lead, H, V)
            st["dS"] = randn(N, H, K, V, dtype=torch.float32, std=0.1) if case["S0"] else None
        if case["op"] == "gd_bwd8":
            st["saved"] = {n: _save8(st.pop(n)) for n in ("q", "k", "v")}
    elif case["op"] == "axes":
        lead = (case["B"], case["T"]) if case["B"] else (case["T"],)
        sections = _sections(case)
        A, R = len(sections), 2 * sum(sections)
        st.update(q=randn(*lead, case["H"], case["D"]), k=randn(*lead, case["Hk"], case["D"]),
                  freqs=10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R),
                  axes=torch.tensor(_pair_axes(sections, case["order"]), dtype=torch.int32, device=dev))
        if case["far"]:
            st["pos"] = torch.randint(0, 1 << 20, (A, *lead), generator=gen, device=dev, dtype=torch.int32)
        else:
            # frames of a clip in raster order: the first axis counts frames of w * w tokens, the others rows and columns
            t = torch.arange(case["T"], device=dev)
            w = 7 + seed % 50
            grid = torch.stack([t // (w * w), t // w % w, t % w][-A:]).int()
            st["pos"] = (grid[:, None] if case["B"] else grid).expand(A, *lead).contiguous()
    else:
        rows, G, C = case["rows"], case["G"], case["C"]
        shape = (rows, G, C) if G > 1 else (rows, C)
        # a residual stream: rows of different sizes, a few channels far above the others
        x = torch.randn(shape, generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device=dev))
        x *= torch.where(torch.rand(C, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        x = x.to(dt)
        if case["op"] == "ckpt":
            st["x"] = x
            return st
        wshape = (G, C) if G > 1 else (C,)
        st.update(saved=_save8(x), w=1.0 + randn(*wshape, dtype=torch.float32, std=0.2),
                  b=randn(*wshape, dtype=torch.float32, std=0.2) if case["center"] else None,
                  z=randn(*shape) if case["gate"] else None, dy=randn(*shape))
    return st


# ------------------------------------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return {"gd_fwd": _gd_fwd, "gd_bwd": _gd_bwd, "gd_bwd8": _gd_bwd, "gd_decode": _gd_decode, "axes": _axes,
            "ckpt": _ckpt, "norm_bwd8": _norm_bwd8}[state["op"]](state)


def _run_own(s):
    import kda_gated_delta_chunk_amd as kda

    c = s["case"]
    dt = DTYPES[c["io"]]
    if s["op"] == "gd_fwd":
        o, S = kda.gd_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s["S0"], cu_seqlens=s["cu"],
                                scale=s["scale"])
        return {"o": o, "S": S}
    if s["op"] in ("gd_bwd", "gd_bwd8"):
        q, k, v = ((kda.Checkpoint8(*s["saved"][n], dt) if s["op"] == "gd_bwd8" else s[n]) for n in ("q", "k", "v"))
        return kda.gd_chunk_bwd(q, k, v, s["g"], s["beta"], s["do"], S0=s["S0"], dS_final=s["dS"], cu_seqlens=s["cu"],
                                scale=s["scale"])
    if s["op"] == "gd_decode":
        o = kda.gd_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], scale=s["scale"])
        return {"o": o, "S": s["S"]}
    if s["op"] == "axes":
        q, k = kda.rotary_axes(s["q"], s["freqs"], s["axes"], s["pos"], k=s["k"], layout=c["layout"],
                               inverse=c["inverse"])
        return {"q": q, "k": k}
    if s["op"] == "ckpt":
        saved = kda.checkpoint8(s["x"])
        return {"x": kda.restore8(saved), "scales": saved.scales}
    return kda.layer_norm_bwd(s["dy"], kda.Checkpoint8(*s["saved"], dt), weight=s["w"], bias=s["b"], o_gate=s["z"],
                              eps=EPS, center=c["center"])


# ---- the gated delta rule: S <- e^g S;  w = beta (v - S^T k);  S <- S + k w^T;  o = scale S^T q
def _inputs(s):
    """q, k, v as the operator takes them: out of their checkpoints where there are any."""
    if "saved" not in s:
        return s["q"], s["k"], s["v"]
    return tuple(_restore8(*s["saved"][n], DTYPES[s["case"]["io"]]) for n in ("q", "k", "v"))


def _blocks(lengths, dev):
    """Token indexes [sequences, blocks * CHUNK] of the sequences, each padded to the longest one's whole blocks, and
    which of them are tokens."""
    n = torch.tensor(lengths, device=dev)
    L = max(1, (max(lengths) + CHUNK - 1) // CHUNK) * CHUNK
    at = torch.arange(L, device=dev)
    valid = at < n[:, None]
    return torch.where(valid, (torch.cumsum(n, 0) - n)[:, None] + at, 0), valid


def _cut(x, idx, valid, H):
    """[B, T, heads, D] as fp32 blocks [N, H, blocks, CHUNK, D], heads repeated to H, zeros where no token is."""
    N, L = idx.shape
    x = x.reshape(-1, x.shape[-2], x.shape[-1])[idx].float() * valid[..., None, None]
    x = x.repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)
    return x.reshape(N, H, L // CHUNK, CHUNK, -1)


def _join(x, idx, valid, shape, dtype, fill=0.0):
    """Blocks [N, H, blocks, CHUNK, D] back to [B, T, heads, D], summed over the v heads that share a q/k head."""
    B, T, heads, D = shape
    N, H = x.shape[:2]
    x = x.reshape(N, heads, H // heads, -1, D).sum(2).transpose(1, 2)
    out = torch.full((B * T, heads, D), fill, dtype=x.dtype, device=x.device)
    out[idx[valid]] = x[valid]
    return out.reshape(B, T, heads, D).to(dtype)


def _chunk_form(s):
    """What both directions need of every block: rows, decays, the pairs' weights and (1 + A)^-1."""
    q, k, v = _inputs(s)
    H = v.shape[2]
    idx, valid = _blocks(s["lengths"], v.device)
    f = dict(shapes=(q.shape, k.shape, v.shape), idx=idx, valid=valid, H=H)
    f["q"], f["k"], f["v"] = (_cut(x, idx, valid, H) for x in (q, k, v))
    f["beta"] = _cut(s["beta"][..., None], idx, valid, H)
    g = _cut(s["g"][..., None], idx, valid, H)[..., 0].double()
    b = torch.cumsum(g, -1)
    i = torch.arange(CHUNK, device=v.device)
    low = i[:, None] >= i
    f["E"] = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -math.inf).float())
    f["strict"] = (i[:, None] > i).float()
    f["enter"], f["leave"] = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    f["total"] = torch.exp(b[..., -1]).float()
    f["kk"] = (f["k"] @ f["k"].transpose(-1, -2)) * f["E"] * f["strict"]
    f["qk"] = (f["q"] @ f["k"].transpose(-1, -2)) * f["E"]
    A = f["beta"] * f["kk"]
    inv = torch.eye(CHUNK, device=v.device).expand(A.shape).clone()
    for r in range(1, CHUNK):
        inv[..., r, :r] = -(A[..., r:r + 1, :r] @ inv[..., :r, :r])[..., 0, :]
    f["inv"] = inv
    return f


def _sweep(s, f):
    """The blocks one after the other: the states before each and at the end, and the rows w that are written."""
    N, H, nb, _, K = f["k"].shape
    U, W = f["inv"] @ (f["beta"] * f["v"]), f["inv"] @ (f["beta"] * f["enter"] * f["k"])
    kl = (f["k"] * f["leave"]).transpose(-1, -2)
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(N, H, K, U.shape[-1], device=U.device)
    states, w = [S], []
    for c in range(nb):
        w.append(U[:, :, c] - W[:, :, c] @ S)
        S = f["total"][:, :, c, None, None] * S + kl[:, :, c] @ w[-1]
        states.append(S)
    return torch.stack(states, 2), torch.stack(w, 2)


def _gd_fwd(s):
    f = _chunk_form(s)
    S, w = _sweep(s, f)
    o = s["scale"] * ((f["enter"] * f["q"]) @ S[:, :, :-1] + f["qk"] @ w)
    return {"o": _join(o, f["idx"], f["valid"], f["shapes"][2], s["v"].dtype), "S": S[:, :, -1].contiguous()}


def _gd_bwd(s):
    f = _chunk_form(s)
    S, w = _sweep(s, f)
    q, k, v, beta, E, strict, enter, leave = (f[n] for n in ("q", "k", "v", "beta", "E", "strict", "enter", "leave"))
    do = s["scale"] * _cut(s["do"], f["idx"], f["valid"], f["H"])
    G = s["dS"] if s["dS"] is not None else torch.zeros_like(S[:, :, 0])
    local, dS_q = f["qk"].transpose(-1, -2) @ do, (enter * q).transpose(-1, -2) @ do
    invT, kl, ke = f["inv"].transpose(-1, -2), leave * k, (enter * k).transpose(-1, -2)
    grads, dw = [], []
    for c in reversed(range(w.shape[2])):
        grads.append(G)
        dw.append(invT[:, :, c] @ (local[:, :, c] + kl[:, :, c] @ G))
        G = f["total"][:, :, c, None, None] * G + dS_q[:, :, c] - ke[:, :, c] @ (beta[:, :, c] * dw[-1])
    grads, dw = torch.stack(grads[::-1], 2), torch.stack(dw[::-1], 2)
    before, after = S[:, :, :-1], S[:, :, 1:]
    read, wread, kept = do @ before.transpose(-1, -2), dw @ before.transpose(-1, -2), w @ grads.transpose(-1, -2)
    dP = (do @ w.transpose(-1, -2)) * E
    M = (dw @ w.transpose(-1, -2)) * strict
    dA = -beta * M * E
    out_q = enter * read + dP @ k
    out_k = dP.transpose(-1, -2) @ q + leave * kept - beta * enter * wread + dA @ k + dA.transpose(-1, -2) @ k
    dbeta = (v * dw).sum(-1) - (enter * k * wread).sum(-1) - (f["kk"] * M).sum(-1)
    # a token's log-decay acts on every pair and state that spans its border: rows' sums less columns' sums after it in
    # the block, and what the block's end passes on
    X = dP * (q @ k.transpose(-1, -2)) - beta * M * f["kk"]
    db = X.sum(-1) - X.sum(-2) + (enter * (q * read - beta * k * wread)).sum(-1) - (leave * k * kept).sum(-1)
    dg = torch.flip(torch.cumsum(torch.flip(db.double(), [-1]), -1), [-1])
    dg = dg + (grads * after).double().sum((-1, -2))[..., None]
    sq, sk, sv = f["shapes"]
    dt, gt, one = s["do"].dtype, s["g"].dtype, sv[:3] + (1,)
    at = (f["idx"], f["valid"])
    return {"dq": _join(out_q, *at, sq, dt), "dk": _join(out_k, *at, sk, dt), "dv": _join(beta * dw, *at, sv, dt),
            "dg": _join(dg[..., None], *at, one, gt)[..., 0], "dbeta": _join(dbeta[..., None], *at, one, gt)[..., 0],
            "dS0": G}


def _gd_decode(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, dim=1)[..., None, :] for n in ("q", "k"))
    S = s["S"].mul_(torch.exp(s["g"].float())[..., None, None])
    w = s["beta"].float()[..., None, None] * (s["v"].float()[..., None, :] - k @ S)
    S += k.transpose(-1, -2) * w
    return {"o": (s["scale"] * (q @ S))[..., 0, :].to(s["v"].dtype), "S": S}


def _axes(s):
    c = s["case"]
    R = 2 * s["freqs"].numel()
    angle = torch.movedim(s["pos"][s["axes"].long()], 0, -1).double() * s["freqs"]
    cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
    if c["inverse"]:
        sin = -sin
    out = {}
    for n in ("q", "k"):
        y = s[n].float()
        a, b = (y[..., :R // 2], y[..., R // 2:R]) if c["layout"] == "half" else (y[..., 0:R:2], y[..., 1:R:2])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
        out[n] = torch.cat([r, y[..., R:]], -1).to(s[n].dtype)
    return out


def _ckpt(s):
    codes, scales = _save8(s["x"])
    return {"x": _restore8(codes, scales, s["x"].dtype), "scales": scales}


def _norm_bwd8(s):
    c = s["case"]
    dt = DTYPES[c["io"]]
    x = _restore8(*s["saved"], dt).float()
    if c["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, dy, out = x * r, s["dy"].float(), {}
    if s["z"] is not None:
        a = torch.sigmoid(s["z"].float())
        y = n * s["w"] + (s["b"] if s["b"] is not None else 0.0)
        out["do_gate"] = (dy * y * a * (1.0 - a)).to(dt)
        dy = dy * a
    out["dweight"] = (dy * n).sum(0)
    if s["b"] is not None:
        out["dbias"] = dy.sum(0)
    d = dy * s["w"]
    dx = d - n * (d * n).mean(-1, keepdim=True)
    if c["center"]:
        dx = dx - d.mean(-1, keepdim=True)
    out["dx"] = (r * dx).to(dt)
    return out


# ------------------------------------------------------------------------------------------------- work
def work(case):
    e, ge = (2 if case[n] == "bf16" else 4 for n in ("io", "gates" if "gates" in case else "io"))
    if case["op"] == "gd_decode":
        N, H, Hk, K, V = (case[n] for n in ("N", "H", "Hk", "K", "V"))
        return {"bytes": 8 * N * H * K * V + 2 * e * N * (Hk * K + H * V) + 2 * ge * N * H, "flops": 7 * N * H * K * V}
    if case["op"].startswith("gd"):
        B, T, H, Hk, K, V = (case[n] for n in ("B", "T", "H", "Hk", "K", "V"))
        states = (case["seqs"] or B) * H * K * V * 4
        nk, nv, gates = B * T * Hk * K, B * T * H * V, 2 * B * T * H * ge
        if case["op"] == "gd_fwd":
            return {"bytes": e * (2 * nk + 2 * nv) + gates + states * (2 if case["S0"] else 1),
                    "flops": 6 * B * T * H * K * V}
        read = e * (2 * nk + nv)
        if case["op"] == "gd_bwd8":
            read = 2 * nk + nv + 4 * B * T * (2 * Hk + H)
        return {"bytes": read + e * (2 * nk + 2 * nv) + 2 * gates + states * (3 if case["S0"] else 1),
                "flops": 16 * B * T * H * K * V}
    if case["op"] == "axes":
        n, A, R = max(case["B"], 1) * case["T"], len(_sections(case)), 2 * sum(_sections(case))
        return {"bytes": 2 * e * n * (case["H"] + case["Hk"]) * case["D"] + 4 * n * A + 6 * R,
                "flops": 3 * n * (case["H"] + case["Hk"]) * R}
    x, w = case["rows"] * case["G"] * case["C"], case["G"] * case["C"] * 4
    scales = 4 * case["rows"] * case["G"] * ((case["C"] + BLOCK - 1) // BLOCK)
    if case["op"] == "ckpt":  # into the checkpoint and out of it
        return {"bytes": 2 * (x * (e + 1) + scales), "flops": 5 * x}
    return {"bytes": x + scales + e * x * (4 if case["gate"] else 2) + 2 * (2 if case["center"] else 1) * w,
            "flops": 17 * x}


# ------------------------------------------------------------------------------------------------- exact
def _by_token(s, bwd):
    """The recurrence token by token in fp64, all sequences at once, some heads at a time; its gradients by the chain
    rule through each token's lines, in reverse."""
    q, k, v = (x.double() for x in _inputs(s))
    dev, f64 = v.device, torch.float64
    B, T, H, V = v.shape
    Hk, K = q.shape[2:]
    n = np.array(s["lengths"])
    N, L = len(n), int(n.max())
    starts = torch.from_numpy(np.cumsum(n) - n).to(dev)
    live = torch.arange(L, device=dev)[:, None] < torch.from_numpy(n).to(dev)  # [L, N]
    at = torch.where(live, starts + torch.arange(L, device=dev)[:, None], 0)
    flat = {"q": q, "k": k, "v": v, "g": s["g"].double()[..., None], "beta": s["beta"].double()[..., None]}
    if bwd:
        flat["do"] = s["do"].double()
    flat = {m: x.reshape(B * T, x.shape[2], x.shape[3]) for m, x in flat.items()}
    res = {"o": torch.zeros(B * T, H, V, dtype=f64, device=dev), "S": torch.zeros(N, H, K, V, dtype=f64, device=dev)}
    if bwd:
        for m, d in (("dq", K), ("dk", K), ("dv", V), ("dg", 1), ("dbeta", 1)):
            res[m] = torch.zeros(B * T, H, d, dtype=f64, device=dev)
        res["dS0"] = torch.zeros_like(res["S"])
    some = max(1, min(H, int(24e9 // (8.0 * K * V * N * max(L, 1))))) if bwd else H
    for h0 in range(0, H, some):
        hs = torch.arange(h0, min(h0 + some, H), device=dev)
        hk = hs // (H // Hk)

        def rows(m, t):  # [N, heads, D], zero where the sequence is over
            x = flat[m][at[t]][:, hk if m in ("q", "k") else hs]
            return x * live[t][:, None, None]

        S = s["S0"][:, hs].double() if s["S0"] is not None else torch.zeros(N, len(hs), K, V, dtype=f64, device=dev)
        kept = []
        for t in range(L):
            kept.append(S if bwd else None)
            kt = rows("k", t)[..., None]
            S = torch.exp(rows("g", t))[..., None] * S
            S = S + kt * (rows("beta", t) * (rows("v", t) - (kt * S).sum(-2)))[..., None, :]
            o = s["scale"] * (rows("q", t)[..., None] * S).sum(-2)
            on = live[t].nonzero()[:, 0]
            res["o"][at[t][on, None], hs] = o[on]
        res["S"][:, hs] = S
        if not bwd:
            continue
        G = s["dS"][:, hs].double() if s["dS"] is not None else torch.zeros_like(S)
        for t in reversed(range(L)):
            qt, kt, vt, do, bt = (rows(m, t) for m in ("q", "k", "v", "do", "beta"))
            a = torch.exp(rows("g", t))[..., None]
            Sd = a * kept.pop()
            err = vt - (kt[..., None] * Sd).sum(-2)
            w = bt * err
            G = G + s["scale"] * qt[..., None] * do[..., None, :]
            dw = (G * kt[..., None]).sum(-2)
            de = bt * dw
            got = {"dq": s["scale"] * ((Sd * do[..., None, :]).sum(-1) + kt * (w * do).sum(-1, keepdim=True)),
                   "dk": (G * w[..., None, :]).sum(-1) - (Sd * de[..., None, :]).sum(-1), "dv": de,
                   "dbeta": (err * dw).sum(-1, keepdim=True)}
            G = G - kt[..., None] * de[..., None, :]
            got["dg"] = (G * Sd).sum((-1, -2))[..., None]
            G = a * G
            on = live[t].nonzero()[:, 0]
            for m, x in got.items():
                res[m][at[t][on, None], hs] = x[on]
        res["dS0"][:, hs] = G
    if not bwd:
        return {"o": res["o"].reshape(v.shape), "S": res["S"]}
    out = {m: res[m].reshape(B, T, Hk, H // Hk, K).sum(3) for m in ("dq", "dk")}
    out.update(dv=res["dv"].reshape(v.shape), dg=res["dg"].reshape(B, T, H), dbeta=res["dbeta"].reshape(B, T, H),
               dS0=res["dS0"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gd_fwd", "gd_bwd", "gd_bwd8"):
        return _by_token(s, case["op"] != "gd_fwd")
    if case["op"] == "gd_decode":
        N, H, K, V = s["S"].shape
        group = H // s["q"].shape[1]
        o, Sn = (torch.empty(sh, dtype=torch.float64, device=s["S"].device) for sh in ((N, H, V), (N, H, K, V)))
        for h in range(H):
            k, q = s["k"][:, h // group].double(), s["q"][:, h // group].double()
            S = torch.exp(s["g"][:, h].double())[:, None, None] * s["S"][:, h]
            e = s["v"][:, h].double() - (k[..., None] * S).sum(1)
            Sn[:, h] = S + s["beta"][:, h].double()[:, None, None] * k[..., None] * e[:, None, :]
            o[:, h] = s["scale"] * (q[..., None] * Sn[:, h]).sum(1)
        return {"o": o, "S": Sn}
    if case["op"] == "axes":
        # e^{i angle} in complex numbers
        pos, axes = s["pos"].cpu().numpy().astype(np.float64), s["axes"].cpu().numpy()
        angle = np.stack([pos[a] * f for a, f in zip(axes, s["freqs"].cpu().numpy())], -1)
        turn = torch.from_numpy(np.exp((-1j if case["inverse"] else 1j) * angle)).to(s["q"].device)[..., None, :]
        out, P = {}, len(axes)
        for n in ("q", "k"):
            y = s[n].double()
            pairs = [(j, j + P) if case["layout"] == "half" else (2 * j, 2 * j + 1) for j in range(P)]
            one, two = (torch.tensor(x, device=y.device) for x in zip(*pairs))
            z = torch.complex(y[..., one], y[..., two]) * turn
            y[..., one], y[..., two] = z.real, z.imag
            out[n] = y
        return out
    if case["op"] == "ckpt":
        # the nearest of the 255 values that a block's step has, block by block
        x, C = s["x"].double(), case["C"]
        y, steps = torch.empty_like(x), []
        for c in range(0, C, BLOCK):
            part = x[..., c:c + BLOCK]
            top = part.abs().amax(-1, keepdim=True)
            y[..., c:c + BLOCK] = torch.round(127 * part / torch.where(top > 0, top, 1.0)) * (top / 127)
            steps.append(top / 127)
        return {"x": y, "scales": torch.cat(steps, -1)}
    codes, scales = s["saved"]
    x = codes.float()
    for c in range(0, case["C"], BLOCK):
        x[..., c:c + BLOCK] *= scales[..., c // BLOCK, None]
    x = x.to(DTYPES[case["io"]]).double()  # the values that the checkpoint stands for are of its type
    mu = x.mean(-1, keepdim=True) if case["center"] else 0.0
    sd = torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + EPS)
    w = s["w"].double()
    b = s["b"].double() if s["b"] is not None else 0.0
    a = 1.0 / (1.0 + torch.exp(-s["z"].double())) if s["z"] is not None else 1.0
    dy, C, out = s["dy"].double(), x.shape[-1], {}
    if s["z"] is not None:
        out["do_gate"] = dy * ((x - mu) / sd * w + b) * a * (1.0 - a)
    # through the standard deviation and the mean, one after the other
    dn = dy * a * w
    dsd = -(dn * (x - mu)).sum(-1, keepdim=True) / sd ** 2
    dc = dn / sd + dsd * (x - mu) / (C * sd)
    out["dx"] = dc - dc.sum(-1, keepdim=True) / C if case["center"] else dc
    out["dweight"] = (dy * a * (x - mu) / sd).sum(0)
    if s["b"] is not None:
        out["dbias"] = (dy * a).sum(0)
    return out
