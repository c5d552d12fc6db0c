"""GPU tests of the gated delta rule with one decay per head against its fp64 definition (oracle.delta).

Tolerances are bounds, element by element: half a step of the result's type relative to the value, and a relative error
that every computed row of the chunk form may carry, times how far the definition lets it carry (``spread``, by the
triangle inequality). A row of fp32 I/O is a sum of up to K + V products, of 32 tokens' rows and of as many weights, each
rounded to 2^-24: (K + V + 128) 2^-24. For bf16 I/O the state as an operand, the pairs' weights and the rows themselves are
pairs of bf16, 2^-17 each, in a chunk's triangular product twice over: 2^-14 covers eight of them.
"""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import delta as od
from oracle import layers as ol
from tests.test_gpu_layers import DT, U, close, half_step, rnd

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def inputs(B, T, H, Hk, K, V, io, seed, gates=None, strength=-3.0, N=None):
    """Keys of about length one, write strengths in (0, 1): the rule contracts."""
    dt, gt = DT[io], DT[gates or io]
    x = dict(q=rnd((B, T, Hk, K), seed, dt), k=rnd((B, T, Hk, K), seed + 1, dt, K ** -0.5),
             v=rnd((B, T, H, V), seed + 2, dt), do=rnd((B, T, H, V), seed + 3, dt),
             g=(-(rnd((B, T, H), seed + 4) + strength).exp()).to(gt), beta=torch.sigmoid(rnd((B, T, H), seed + 7)).to(gt))
    n = B if N is None else N
    x["S0"], x["dS"] = rnd((n, H, K, V), seed + 5, std=0.5), rnd((n, H, K, V), seed + 6, std=0.5)
    return x


ARGS = ("q", "k", "v", "g", "beta")


def carried(x):
    """The relative error of a computed row."""
    K, V = x["q"].shape[-1], x["v"].shape[-1]
    return (K + V + 128) * U if x["q"].dtype is torch.float32 else 2.0 ** -14


def check_fwd(x, o, S, cu=None, scale=1.0, S0=True):
    ro, rS, so, sS = od.gd_forward(*(x[n] for n in ARGS), x["S0"] if S0 else None, cu, scale, spread=True)
    live = ~ro.isnan()
    close("o", o.cpu()[live], ro[live], (half_step(o.dtype) * ro.abs() + carried(x) * so)[live])
    close("S_final", S, rS, (U * rS.abs() + carried(x) * sS).expand_as(rS))


def check_bwd(x, r, cu=None, scale=1.0, S0=True, dS=True, names=("dq", "dk", "dv", "dg", "dbeta", "dS0")):
    ref, far = od.gd_backward(*(x[n] for n in ARGS), x["do"], x["S0"] if S0 else None, x["dS"] if dS else None, cu, scale,
                              spread=True)
    group = x["v"].shape[2] // x["q"].shape[2]
    for n in names:
        if n not in r:
            continue
        live = ~ref[n].isnan()
        tol = half_step(r[n].dtype) * ref[n].abs() + (carried(x) + group * U) * far[n]
        close(n, r[n].cpu()[live], ref[n][live], tol[live])


SIZES = [  # B, T, H, Hk, K, V
    (1, 1, 1, 1, 32, 32), (2, 5, 3, 3, 64, 32), (1, 31, 2, 1, 32, 64), (1, 32, 2, 2, 128, 128), (2, 65, 4, 2, 64, 128),
    (1, 130, 6, 2, 128, 64), (1, 33, 9, 3, 128, 32), (1, 300, 2, 2, 32, 128), (1, 257, 8, 1, 64, 64), (3, 97, 1, 1, 128, 128),
]


@pytest.mark.parametrize("io,gates", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("B,T,H,Hk,K,V", SIZES)
def test_fwd_and_bwd(B, T, H, Hk, K, V, io, gates):
    x = inputs(B, T, H, Hk, K, V, io, 100 + T, gates)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], scale=0.3)
    check_fwd(x, o, S, scale=0.3)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], scale=0.3)
    assert set(r) == {"dq", "dk", "dv", "dg", "dbeta", "dS0"}
    assert r["dg"].dtype is DT[gates] and r["dbeta"].dtype is DT[gates] and r["dq"].dtype is DT[io]
    check_bwd(x, r, scale=0.3)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_errors_of_long_sums(io):
    """2-norms: rounding errors that are independent of each other stay below the bound of one pair of bf16 (fp32 I/O: of
    16 roundings), however many tokens they are summed over; dg and dbeta in fp32 are sums with cancellation, four times."""
    x = inputs(1, 700, 4, 2, 128, 128, io, 17, "fp32")
    one = 2.0 ** -17 if io == "bf16" else 16 * U
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    _, rS = od.gd_forward(*(x[n] for n in ARGS), x["S0"])
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    ref = od.gd_backward(*(x[n] for n in ARGS), x["do"], x["S0"], x["dS"])
    assert float((S.cpu().double() - rS).norm() / rS.norm()) < one
    assert float((r["dS0"].cpu().double() - ref["dS0"]).norm() / ref["dS0"].norm()) < one
    for n in ("dg", "dbeta"):
        assert float((r[n].cpu().double() - ref[n]).norm() / ref[n].norm()) < 4 * one, n


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_without_states(io):
    x = inputs(1, 100, 2, 2, 64, 64, io, 7)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS))
    check_fwd(x, o, S, S0=False)
    o2, none = kda.gd_chunk_fwd(*(x[n] for n in ARGS), output_final_state=False)
    assert none is None and torch.equal(o, o2)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], want_dS0=False)
    assert set(r) == {"dq", "dk", "dv", "dg", "dbeta"}
    check_bwd(x, r, S0=False, dS=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [255, 256, 257, 513, 1100])
def test_segments_of_the_gradients(io, T):
    x = inputs(1, T, 2, 1, 64, 32, io, 11)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    check_bwd(x, r)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("strength", [-20.0, 0.0, 1.5])
@pytest.mark.parametrize("T", [31, 64, 97])
def test_decays_from_none_to_strong(io, strength, T):
    x = inputs(1, T, 2, 1, 64, 64, io, 14, strength=strength)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    check_fwd(x, o, S)
    check_bwd(x, kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"]))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_tokens_that_clear_or_do_not_write(io):
    """-inf and beyond fp32's exponent clear the state; beta = 0 writes nothing (nothing is divided by it); beta = 1."""
    x = inputs(1, 200, 4, 4, 64, 32, io, 51)
    x["g"][:, 10::37, 0] = -INF
    x["g"][:, 5::20, 1] = -1000.0
    x["g"][:, :, 2] = 0.0
    x["beta"][:, 3::5, 1] = 0.0
    x["beta"][:, :, 2] = 0.0
    x["beta"][:, :, 3] = 1.0
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    check_fwd(x, o, S)
    assert torch.equal(S[0, 2], x["S0"][0, 2])
    check_bwd(x, kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"]))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_the_same_key_again_and_again(io):
    """One key of length one for all tokens, beta = 1: every token overwrites the one before it, and the chunk's inverse
    has entries of size one throughout."""
    x = inputs(1, 70, 1, 1, 32, 32, "fp32", 55, strength=-20.0)
    key = torch.zeros(32)
    key[3] = 1.0
    x["k"] = key.cuda().expand(1, 70, 1, 32).contiguous()
    x["beta"][:] = 1.0
    x = {n: t.to(DT[io]) if n not in ("S0", "dS") else t for n, t in x.items()}
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    check_fwd(x, o, S)
    # what the key holds is the last token's value
    close("S row", S[0, 0, 3], ol.f64(x["v"])[0, -1, 0], torch.full((32,), 2.0 ** -13 * float(x["v"].abs().max())).double())
    check_bwd(x, kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"]))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", [[0, 0, 1, 64, 64, 191, 400], [3, 700, 700, 1180], [0, 1180], [1180, 1180], [0, 0]])
def test_packed(io, cu):
    """Empty sequences, one token, borders inside a chunk, segments; rows outside the sequences stay as they were and
    are not read."""
    T, N = 1200, len(cu) - 1
    x = inputs(1, T, 4, 2, 32, 64, io, 21, N=N)
    out = torch.ones(T, dtype=torch.bool)
    out[cu[0]:cu[-1]] = False
    for n in (*ARGS, "do"):
        x[n][:, out.cuda()] = NAN
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], cu_seqlens=c, out=o)
    assert bool((o[:, out.cuda()] == 7.0).all())
    check_fwd(x, o, S, cu=c.cpu())
    res = {"d" + n: torch.full_like(x[n], 7.0) for n in ARGS}
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c, out=res)
    for n in res:
        assert r[n] is res[n] and bool((r[n][:, out.cuda()] == 7.0).all()), n
    check_bwd(x, r, cu=c.cpu())


def test_many_packed_sequences():
    """More sequences than the table kernel takes at a time, most of them empty or of one token."""
    N, T = 2500, 3000
    gen = torch.Generator().manual_seed(3)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, 2, (N - 1,), generator=gen).cumsum(0),
                    torch.tensor([T])])
    x = inputs(1, T, 1, 1, 32, 32, "bf16", 31, N=N)
    c = cu.to(torch.int32).cuda()
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], cu_seqlens=c)
    check_fwd(x, o, S, cu=c.cpu())
    check_bwd(x, kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c), cu=c.cpu())


def test_corrupt_cu_seqlens_stay_in_bounds():
    """Entries out of range or falling are clamped and made non-decreasing, as the oracle reads them."""
    x = inputs(1, 300, 2, 2, 32, 32, "bf16", 41, N=5)
    c = torch.tensor([-5, 100, 40, 2 ** 31 - 1, 7, 250], dtype=torch.int32, device="cuda")
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], cu_seqlens=c)
    check_fwd(x, o, S, cu=c.cpu())
    check_bwd(x, kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c), cu=c.cpu())


def test_empty():
    x = inputs(2, 0, 2, 1, 32, 32, "fp32", 61)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    assert o.shape == (2, 0, 2, 32) and torch.equal(S, x["S0"])
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], dS_final=x["dS"])
    assert torch.equal(r["dS0"], x["dS"]) and r["dg"].shape == (2, 0, 2)
    assert bool((kda.gd_chunk_fwd(*(x[n] for n in ARGS))[1] == 0).all())


def test_deterministic_whatever_the_workspace_held():
    x = inputs(1, 900, 2, 1, 128, 64, "bf16", 71)
    wf = torch.empty(kda.gd_workspace_bytes(1, 900, 2, 128, 64, 1, Hk=1), dtype=torch.uint8, device="cuda")
    wb = torch.empty(kda.gd_bwd_workspace_bytes(1, 900, 2, 128, 64, 1, Hk=1), dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0, 255):
        wf.fill_(fill), wb.fill_(fill)
        o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], workspace=wf)
        r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], workspace=wb)
        got = {"o": o, "S": S, **r}
        if first is not None:
            for n in got:
                assert torch.equal(got[n], first[n]), n
        first = got


def test_with_one_decay_for_all_channels_it_is_kda():
    """The package's own recurrence with a decay per key channel, given the same number for each."""
    x = inputs(2, 150, 3, 3, 128, 128, "fp32", 75, strength=-4.0)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    g = x["g"][..., None].expand(2, 150, 3, 128).contiguous()
    ko, kS = kda.chunk_fwd(x["q"], x["k"], x["v"], g, x["beta"], S0=x["S0"])
    assert float((o - ko).abs().max()) < 1e-4 * float(ko.square().mean().sqrt())
    assert float((S - kS).abs().max()) < 1e-4 * float(kS.square().mean().sqrt())


def test_a_sequence_in_two_calls():
    """The state that one call ends with starts the next; the same for the gradients, from the other end."""
    x = inputs(1, 300, 4, 2, 64, 64, "fp32", 77)
    P = 141
    cut = lambda a, b: [x[n][:, a:b].contiguous() for n in ARGS]  # noqa: E731
    o1, S1 = kda.gd_chunk_fwd(*cut(0, P), S0=x["S0"])
    o2, S2 = kda.gd_chunk_fwd(*cut(P, 300), S0=S1)
    check_fwd(x, torch.cat([o1, o2], 1), S2)
    b = kda.gd_chunk_bwd(*cut(P, 300), x["do"][:, P:].contiguous(), S0=S1, dS_final=x["dS"])
    a = kda.gd_chunk_bwd(*cut(0, P), x["do"][:, :P].contiguous(), S0=x["S0"], dS_final=b["dS0"])
    check_bwd(x, {**{n: torch.cat([a[n], b[n]], 1) for n in ("dq", "dk", "dv", "dg", "dbeta")}, "dS0": a["dS0"]})


@pytest.mark.parametrize("io,gates", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("N,H,Hk,K,V", [(1, 1, 1, 32, 32), (3, 6, 2, 128, 64), (7, 5, 5, 64, 128), (2, 4, 1, 32, 128),
                                        (5, 3, 1, 128, 32), (130, 8, 8, 128, 128), (700, 8, 8, 32, 64)])
def test_decode(N, H, Hk, K, V, io, gates):
    dt, gt = DT[io], DT[gates]
    q, k, v = rnd((N, Hk, K), 1, dt), rnd((N, Hk, K), 2, dt, K ** -0.5), rnd((N, H, V), 3, dt)
    g, beta = (-(rnd((N, H), 4) - 2.0).exp()).to(gt), torch.sigmoid(rnd((N, H), 6)).to(gt)
    S = rnd((N, H, K, V), 5)
    g[0, 0] = -INF
    ro, rS = od.gd_step(q, k, v, g, beta, S, 0.5)
    # every term by its absolute value: e^g S (1 + beta |k| |k|^T) + beta |k| |v|^T
    a = {n: ol._expand(ol.f64(t).abs(), H) for n, t in (("q", q), ("k", k))}
    aS = torch.exp(ol.f64(g))[..., None, None] * ol.f64(S).abs()
    w = ol.f64(beta)[..., None] * (ol.f64(v).abs() + (a["k"][..., None] * aS).sum(2))
    full = aS + a["k"][..., None] * w[:, :, None]
    ao = 0.5 * ((a["q"][..., None] * aS).sum(2) + (a["q"] * a["k"]).sum(-1, keepdim=True) * w)
    o = kda.gd_decode_step(q, k, v, g, beta, S, scale=0.5)
    close("S", S, rS, (K + 16) * U * full)
    close("o", o, ro, half_step(dt) * ro.abs() + 2 * (K + 16) * U * ao)


def test_prefill_then_decode_is_the_whole_sequence():
    x = inputs(2, 150, 4, 2, 64, 64, "fp32", 81)
    P = 131
    head, S = kda.gd_chunk_fwd(*[x[n][:, :P].contiguous() for n in ARGS], S0=x["S0"])
    outs = [head]
    for t in range(P, 150):
        outs.append(kda.gd_decode_step(*[x[n][:, t].contiguous() for n in ARGS], S)[:, None])
    check_fwd(x, torch.cat(outs, 1), S)


# ------------------------------------------------------------------------------------------ values that are not finite
def finite_agree(name, got, ref, far, x):
    """Where the definition's result is finite: close to it."""
    got = got.cpu()
    live = ref.isfinite() & far.isfinite()
    close(name, got[live], ref[live], (half_step(got.dtype) * ref.abs() + carried(x) * far)[live])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [32, 61, 100])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("q", -INF), ("g", NAN), ("beta", INF)])
@pytest.mark.parametrize("at", [0, 7, 15, 16, 31])
def test_forward_is_causal(at, name, value, T, io):
    """One such entry at a token of the last chunk: the outputs before it, and of other columns, do not see it."""
    x = inputs(1, T, 2, 2, 64, 64, io, 500 + T)
    t = min((T - 1) // 32 * 32 + at, T - 1)
    clean, _, far, _ = od.gd_forward(*(x[n] for n in ARGS), x["S0"], spread=True)
    if name in ("g", "beta"):
        x[name][0, t, 1] = value
    else:
        x[name][0, t, 1, 37] = value
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    ref, rS = od.gd_forward(*(x[n] for n in ARGS), x["S0"])
    finite_agree("o before", o[:, :t], clean[:, :t], far[:, :t], x)
    finite_agree("the other head", o[:, :, 0], clean[:, :, 0], far[:, :, 0], x)
    bad = ~ref.isfinite()
    finite_agree("o", o[~bad], clean[~bad], far[~bad], x)
    assert bool(bad.any()) and not bool(o.cpu()[bad].isfinite().any())
    assert bool(S[0, 0].isfinite().all()) and torch.equal(S[0, 1].isfinite().cpu(), rS[0, 1].isfinite())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(32, 128), (128, 32), (128, 128)])
def test_garbage_behind_a_prompt(K, V, io):
    """Prompts of several lengths in rows of one batch, garbage behind them: their outputs are those of clean rows."""
    T, lengths = 200, [5, 32, 47, 170]
    x = inputs(4, T, 3, 1, K, V, io, 600)
    ref, _, far, _ = od.gd_forward(*(x[n] for n in ARGS), x["S0"], spread=True)
    for b, n in enumerate(lengths):
        for name in ARGS:
            x[name][b, n:] = NAN if b % 2 else INF
    o, _ = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    for b, n in enumerate(lengths):
        finite_agree("o", o[b, :n], ref[b, :n], far[b, :n], x)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [32, 61, 100])
@pytest.mark.parametrize("name,value", [("v", NAN), ("k", INF), ("q", NAN), ("do", NAN), ("do", -INF)])
@pytest.mark.parametrize("at", [0, 7, 16, 31])
def test_gradients_reach_what_depends(at, name, value, T, io):
    """dq sees k and v up to its token, dv sees no v, dk and dv see q and do from theirs on; dg and dbeta are summed over
    a head's tokens and may be spoiled throughout."""
    x = inputs(1, T, 2, 2, 64, 64, io, 700 + T)
    t = min((T - 1) // 32 * 32 + at, T - 1)
    clean, far = od.gd_backward(*(x[n] for n in ARGS), x["do"], x["S0"], x["dS"], spread=True)
    x[name][0, t, 1, 37] = value
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        finite_agree(n + " of the other head", r[n][:, :, 0], clean[n][:, :, 0], far[n][:, :, 0], x)
    if name in ("v", "k"):
        finite_agree("dq", r["dq"][:, :t], clean["dq"][:, :t], far["dq"][:, :t], x)
    if name == "v":
        finite_agree("dk", r["dk"][:, :t], clean["dk"][:, :t], far["dk"][:, :t], x)
        finite_agree("dv", r["dv"], clean["dv"], far["dv"], x)
    else:
        for n in ("dk", "dv"):
            finite_agree(n, r[n][:, t + 1:], clean[n][:, t + 1:], far[n][:, t + 1:], x) if name != "k" else None
    if name in ("q", "do"):
        finite_agree("dq", r["dq"][:, t + 1:], clean["dq"][:, t + 1:], far["dq"][:, t + 1:], x)
        finite_agree("dq", r["dq"][:, :t], clean["dq"][:, :t], far["dq"][:, :t], x)


# ------------------------------------------------------------------------------------------ streams, graphs, offsets
def test_two_graphs_replayed_in_turn():
    """A forward and a backward call captured with workspaces of their own, replayed with eager work between, against
    the eager results."""
    x = inputs(1, 333, 4, 2, 64, 64, "bf16", 91)
    eager_o, eager_S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    eager_r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    torch.cuda.synchronize()
    f, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(f):
        o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    with torch.cuda.graph(b):
        r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    for _ in range(3):
        o.zero_(), S.zero_()
        for t in r.values():
            t.zero_()
        f.replay()
        b.replay()
        other = kda.gd_chunk_fwd(*(x[n] for n in ARGS))[0]
        torch.cuda.synchronize()
        assert torch.equal(o, eager_o) and torch.equal(S, eager_S) and not torch.equal(other, o)
        for n in r:
            assert torch.equal(r[n], eager_r[n]), n


def test_on_a_stream_of_its_own():
    x = inputs(1, 500, 8, 4, 128, 128, "bf16", 95)
    ref = kda.gd_chunk_fwd(*(x[n] for n in ARGS))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = [x[n].clone() for n in ARGS]  # on this stream: the call has to follow it
        got = kda.gd_chunk_fwd(*late)
        S = got[1].clone()
        step = kda.gd_decode_step(*[t[:, -1].contiguous() for t in late], S)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and bool(step.isfinite().all())


def test_long_offsets():
    """Elements past 2^31: the last packed sequences of a batch equal the same sequences alone, bit for bit (their chunks
    start where the sequences do)."""
    H, K = 96, 128
    T = (1 << 31) // (H * K) + 5000
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = [torch.empty((1, T, H, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3)]
    k *= K ** -0.5
    g = -torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    beta = torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    cu = torch.tensor([0, T - 4096, T - 77, T], dtype=torch.int32, device="cuda")
    o, S = kda.gd_chunk_fwd(q, k, v, g, beta, cu_seqlens=cu, scale=0.1)
    for n, (a, b) in enumerate([(T - 4096, T - 77), (T - 77, T)]):
        o1, S1 = kda.gd_chunk_fwd(*[t[:, a:b].contiguous() for t in (q, k, v, g, beta)], scale=0.1)
        assert torch.equal(o[:, a:b], o1) and torch.equal(S[n + 1], S1[0])


def test_gradients_at_long_offsets():
    H, K = 96, 128
    T = (1 << 31) // (H * K) + 5000
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v, do = [torch.empty((1, T, H, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4)]
    k *= K ** -0.5
    g = -torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    beta = torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    cu = torch.tensor([0, T - 4096, T - 77, T], dtype=torch.int32, device="cuda")
    r = kda.gd_chunk_bwd(q, k, v, g, beta, do, cu_seqlens=cu, scale=0.1)
    for n, (a, b) in enumerate([(T - 4096, T - 77), (T - 77, T)]):
        r1 = kda.gd_chunk_bwd(*[t[:, a:b].contiguous() for t in (q, k, v, g, beta, do)], scale=0.1)
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(r[name][:, a:b], r1[name]), name
        assert torch.equal(r["dS0"][n + 1], r1["dS0"][0])


@pytest.mark.parametrize("io,K", [("bf16", 128), ("bf16", 32), ("fp32", 128), ("fp32", 64)])
def test_many_heads_share_compute_units(io, K):
    """Where there are more column tiles than compute units both of a head go to one workgroup: the same bits as of a call of
    few heads (two chunks, so that the gradients' segments are the same)."""
    H, Hk, V = 260, 130, 128
    x = inputs(1, 45, H, Hk, K, V, io, 97)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], scale=0.3)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], scale=0.3)
    for h in (0, 126, 256):
        few = {n: t[:, :, h // 2:h // 2 + 2] if n in ("q", "k") else t[:, h:h + 4] if n in ("S0", "dS") else t[:, :, h:h + 4]
               for n, t in x.items()}
        few = {n: t.contiguous() for n, t in few.items()}
        o1, S1 = kda.gd_chunk_fwd(*(few[n] for n in ARGS), S0=few["S0"], scale=0.3)
        r1 = kda.gd_chunk_bwd(*(few[n] for n in ARGS), few["do"], S0=few["S0"], dS_final=few["dS"], scale=0.3)
        assert torch.equal(o[:, :, h:h + 4], o1) and torch.equal(S[:, h:h + 4], S1)
        for n in ("dv", "dg", "dbeta"):
            assert torch.equal(r[n][:, :, h:h + 4], r1[n]), n
        for n in ("dq", "dk"):
            assert torch.equal(r[n][:, :, h // 2:h // 2 + 2], r1[n]), n
        assert torch.equal(r["dS0"][:, h:h + 4], r1["dS0"])


def test_many_packed_sequences_share_compute_units():
    """The same for packed ones, whose workgroups start in the order of their lengths: each as if it were alone."""
    H, K, V, N = 32, 64, 128, 41
    gen = torch.Generator().manual_seed(12)
    lengths = torch.randint(0, 90, (N,), generator=gen)
    lengths[5] = lengths[17] = 0
    lengths[23] = 700
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)]).to(torch.int32)
    T = int(cu[-1])
    x = inputs(1, T, H, H // 2, K, V, "bf16", 98, gates="fp32", N=N)
    dev = cu.cuda()
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], cu_seqlens=dev)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=dev)
    assert torch.equal(S[5], x["S0"][5]) and torch.equal(r["dS0"][17], x["dS"][17])
    for n in (0, 6, 23, 40):
        a, b = int(cu[n]), int(cu[n + 1])
        one = [x[m][:, a:b].contiguous() for m in ARGS + ("do",)]
        S0, dS = x["S0"][n:n + 1].contiguous(), x["dS"][n:n + 1].contiguous()
        o1, S1 = kda.gd_chunk_fwd(*one[:5], S0=S0)
        r1 = kda.gd_chunk_bwd(*one, S0=S0, dS_final=dS)
        assert torch.equal(o[:, a:b], o1) and torch.equal(S[n:n + 1], S1)
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(r[m][:, a:b], r1[m]), m
        assert torch.equal(r["dS0"][n:n + 1], r1["dS0"])


@pytest.mark.parametrize("N", [1023, 1024, 1025, 2500])
def test_many_short_sequences(N):
    """Packed sequences of two tokens equal the rows of a batch, bit for bit, also where the table takes several turns."""
    x = inputs(N, 2, 2, 1, 32, 64, "bf16", 99)
    flat = {n: x[n].reshape((1, 2 * N) + x[n].shape[2:]) for n in ARGS + ("do",)}
    cu = torch.arange(0, 2 * N + 1, 2, dtype=torch.int32, device="cuda")
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    po, pS = kda.gd_chunk_fwd(*(flat[n] for n in ARGS), S0=x["S0"], cu_seqlens=cu)
    assert torch.equal(po.reshape(o.shape), o) and torch.equal(pS, S)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    pr = kda.gd_chunk_bwd(*(flat[n] for n in ARGS), flat["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=cu)
    for n in r:
        assert torch.equal(pr[n].reshape(r[n].shape), r[n]), n


def test_refusals():
    x = inputs(1, 8, 4, 2, 32, 32, "bf16", 93)
    q, k, v, g, beta = (x[n] for n in ARGS)
    with pytest.raises(ValueError):
        kda.gd_chunk_fwd(q[:, ::2], k, v, g, beta)
    with pytest.raises(ValueError, match="contiguous"):
        kda.gd_chunk_fwd(q, k, torch.empty(1, 8, 32, 4, device="cuda", dtype=torch.bfloat16).transpose(2, 3), g, beta)
    with pytest.raises(TypeError):
        kda.gd_chunk_fwd(q, k, v, g.float(), beta)  # both gates of one type
    with pytest.raises(TypeError):
        kda.gd_chunk_fwd(q, k, v, g.half(), beta)
    with pytest.raises(ValueError):
        kda.gd_chunk_fwd(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous(), beta[:, :, :3].contiguous())
    with pytest.raises(ValueError):
        kda.gd_chunk_bwd(q, k, v, g, beta, x["do"], out={"dS": g})
    with pytest.raises(ValueError):
        kda.gd_chunk_bwd(q, k, v, g, beta, x["do"], want_dS0=False, out={"dS0": x["S0"]})
    with pytest.raises(kda.KDAError):
        kda.gd_chunk_fwd(*[torch.zeros(1, 8, 4, 48, device="cuda") for _ in range(3)],
                         *[torch.zeros(1, 8, 4, device="cuda") for _ in range(2)])
    with pytest.raises(kda.KDAError):
        kda.gd_chunk_fwd(q, k, v, g, beta, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    off = torch.zeros(q.numel() + 1, device="cuda", dtype=q.dtype)[1:].view(q.shape)  # 2 bytes behind a 16-byte border
    with pytest.raises(kda.KDAError):
        kda.gd_chunk_fwd(off, k, v, g, beta)
    with pytest.raises(kda.KDAError):
        kda.gd_chunk_fwd(q, k, v, g, beta, out=v)  # the result may not be an input
    S = torch.zeros(8, 4, 32, 32, device="cuda")
    with pytest.raises(ValueError):
        kda.gd_decode_step(q[0], k[0], v[0], g[0], beta[0], S[:7])
    with pytest.raises(kda.KDAError):
        kda.gd_decode_step(q[0], k[0], v[0], g[0], beta[0], S, out=v[0])
