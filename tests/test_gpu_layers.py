"""GPU tests of the operators around the recurrence against their fp64 definitions (oracle.layers).

Tolerances are bounds, element by element. A sum of n products in fp32 is off by at most about n 2^-24 of the sum of
the products' absolute values; that sum is the same definition evaluated on absolute values (every term of the linear
attention and its gradients is a product with positive weights). On top come half a step of the result's type,
relative to the value, and, for bf16, the operands that the kernels round: the fp32 state read as a bf16 operand, half a
step (2^-8) of the sum of absolute values. Results in fp32 of bf16 inputs (states) have no rounded operand.
"""
import math

import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import layers as ol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24  # half a step of fp32


def rnd(shape, seed, dt=torch.float32, std=1.0):
    x = std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    return x.to(dt).cuda()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def close(name, x, ref, tol):
    """|x - ref| <= tol everywhere, and x finite where ref is."""
    x = x.detach().to("cpu", torch.float64)
    assert x.shape == ref.shape, (name, x.shape, ref.shape)
    bad = ~((x - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        name, int(bad.sum()), bad.numel(), float(((x - ref).abs() / tol.clamp(min=1e-300)).nan_to_num(nan=1e9).max()))


# ------------------------------------------------------------------------------- linear attention, one decay per head
def hd_inputs(B, T, H, Hk, K, V, io, seed, decay="token", strength=-3.0, N=None):
    dt = DT[io]
    x = dict(q=rnd((B, T, Hk, K), seed, dt), k=rnd((B, T, Hk, K), seed + 1, dt, K ** -0.5), v=rnd((B, T, H, V), seed + 2, dt),
             do=rnd((B, T, H, V), seed + 3, dt))
    g = -(rnd((B, T, H) if decay == "token" else (H,), seed + 4) + strength).exp()
    x["g"] = g.to(dt) if decay == "token" else g
    n = B if N is None else N
    x["S0"], x["dS"] = rnd((n, H, K, V), seed + 5, std=0.5), rnd((n, H, K, V), seed + 6, std=0.5)
    return x


def _abs(x):
    return {n: t.abs() if n != "g" else t for n, t in x.items()}


def _roundings(T, K, V):
    """Roundings on a term's way into a result: its dot product, its weight (exponent, exponential, product: 16), its
    sum inside the chunk and over the chunks (64 tokens, then one multiplication and one addition per chunk)."""
    return K + V + 64 + 2 * (T // 32 + 1) + 16


def check_fwd(x, o, S, cu=None, scale=1.0, S0=True):
    dt = x["q"].dtype
    args = [x[n] for n in ("q", "k", "v", "g")]
    ao, aS = ol.hd_forward(*[_abs(x)[n] for n in ("q", "k", "v", "g")], x["S0"].abs() if S0 else None, cu, abs(scale))
    ro, rS = ol.hd_forward(*args, x["S0"] if S0 else None, cu, scale)
    T, K, V = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    n = _roundings(T, K, V)
    op = half_step(dt) if dt != torch.float32 else 0.0
    live = ~ro.isnan()
    close("o", o.cpu()[live], ro[live], (half_step(dt) * ro.abs() + (op + n * U) * ao)[live])
    close("S_final", S, rS, n * U * aS)


def check_bwd(x, r, cu=None, scale=1.0, S0=True, dS=True, decay="token"):
    dt = x["q"].dtype
    a = _abs(x)
    ref = ol.hd_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"] if S0 else None, x["dS"] if dS else None, cu,
                         scale)
    mag = ol.hd_backward(a["q"], a["k"], a["v"], a["g"], a["do"], a["S0"] if S0 else None, a["dS"] if dS else None, cu,
                         abs(scale))
    T, K, V = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    n = _roundings(T, K, V) + x["v"].shape[2] // x["q"].shape[2]
    op = half_step(dt) if dt != torch.float32 else 0.0
    for name in ("dq", "dk", "dv"):
        live = ~ref[name].isnan()
        close(name, r[name].cpu()[live], ref[name][live],
              (half_step(dt) * ref[name].abs() + (op + n * U) * mag[name])[live])
    if "dS0" in r:
        close("dS0", r["dS0"], ref["dS0"], n * U * mag["dS0"])
    if decay == "token":
        # dg is summed from the rows' do.o less v.dv behind a token: its bound is that of those sums. For bf16 the
        # state is a pair of bf16 here (2^-16 of its terms), and so are the weighted products.
        ao, _ = ol.hd_forward(a["q"], a["k"], a["v"], a["g"], a["S0"] if S0 else None, cu, abs(scale))
        parts = (ol.f64(a["do"]) * ao).sum(-1) + (ol.f64(a["v"]) * mag["dv"]).sum(-1)
        tol = torch.zeros_like(parts).reshape(-1, parts.shape[-1])
        flat = parts.reshape(-1, parts.shape[-1])
        _, aS = ol.hd_forward(a["q"], a["k"], a["v"], a["g"], a["S0"] if S0 else None, cu, abs(scale))
        for i, (t0, t1) in enumerate(ol._seqs(*x["q"].shape[:2], cu)):
            tail = (aS[i] * a["dS"][i].cpu().double()).sum((1, 2)) if dS else 0.0
            tol[t0:t1] = flat[t0:t1].flip(0).cumsum(0).flip(0) + tail
        live = ~ref["dg"].isnan()
        pair = 2.0 ** -15 if dt != torch.float32 else 0.0
        close("dg", r["dg"].cpu()[live], ref["dg"][live],
              (half_step(dt) * ref["dg"].abs() + (pair + n * U) * tol.reshape(parts.shape))[live])


SIZES = [  # B, T, H, Hk, K, V
    (1, 1, 1, 1, 32, 32), (2, 5, 3, 3, 64, 32), (1, 63, 2, 1, 32, 64), (1, 64, 2, 2, 128, 128), (2, 65, 4, 2, 64, 128),
    (1, 130, 6, 2, 128, 64), (1, 33, 9, 3, 128, 32), (1, 300, 2, 2, 32, 128), (1, 257, 8, 1, 64, 64),
]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,T,H,Hk,K,V", SIZES)
def test_hd_fwd_and_bwd(B, T, H, Hk, K, V, io, decay):
    x = hd_inputs(B, T, H, Hk, K, V, io, 100 + T, decay)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], scale=0.3)
    check_fwd(x, o, S, scale=0.3)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], scale=0.3)
    assert set(r) == {"dq", "dk", "dv", "dS0"} | ({"dg"} if decay == "token" else set())
    check_bwd(x, r, scale=0.3, decay=decay)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_hd_without_states(io):
    x = hd_inputs(1, 100, 2, 2, 64, 64, io, 7)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    check_fwd(x, o, S, S0=False)
    o2, none = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=False)
    assert none is None and torch.equal(o, o2)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], want_dS0=False, want_dg=False)
    assert set(r) == {"dq", "dk", "dv"}
    check_bwd(x, {**r, "dg": kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"])["dg"]}, S0=False, dS=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [600, 1537, 4100, 9000])
def test_hd_segments(io, T):
    """One head over many tokens runs as segments, few or many: the same results."""
    x = hd_inputs(1, T, 1, 1, 64, 64, io, 11)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    check_fwd(x, o, S)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"])
    check_bwd(x, r)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,Hk,K,V", [(2100, 2, 1, 128, 128), (1500, 3, 1, 128, 32), (1501, 1, 1, 32, 128),
                                        (1100, 5, 5, 32, 32)])
def test_hd_segments_of_shared_heads(io, T, H, Hk, K, V):
    x = hd_inputs(1, T, H, Hk, K, V, io, 12)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    check_fwd(x, o, S)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"])
    check_bwd(x, r)
    cu = [5, 1, T - 700, T - 699, T - 3]  # falls once: read as 5
    x = hd_inputs(1, T, H, Hk, K, V, io, 13, N=4)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=c)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c)
    for res in (o, r["dq"], r["dk"], r["dv"], r["dg"]):  # rows of no sequence are as they were: anything
        res[:, :5], res[:, T - 3:] = 0.0, 0.0
    check_fwd(x, o, S, cu=c.cpu())
    check_bwd(x, r, cu=c.cpu())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("strength", [-20.0, -1.0, 0.0, 1.5])
@pytest.mark.parametrize("T", [31, 32, 95, 96, 97, 161])
def test_hd_lengths_about_whole_chunks(io, strength, T):
    """One to six chunks, full and ragged, with decays from none to e^-200 a chunk, so that two chunks' decays are
    within one scaling, or only one's, or neither's."""
    x = hd_inputs(1, T, 2, 1, 64, 64, io, 14, strength=strength)
    x["g"][:, : T // 2, 1] *= 0.25
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    check_fwd(x, o, S)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"])
    check_bwd(x, r)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_hd_nan_stays_in_its_sequence_and_head(io):
    """A NaN reaches its own head of its own sequence, and no token before its chunk of 32."""
    cu = torch.tensor([0, 40, 150, 190], dtype=torch.int32, device="cuda")
    x = hd_inputs(1, 190, 3, 3, 64, 64, io, 15, N=3)
    args = [x[n] for n in ("q", "k", "v", "g")]
    o, S = kda.hd_chunk_fwd(*args, S0=x["S0"], cu_seqlens=cu)
    r = kda.hd_chunk_bwd(*args, x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=cu)
    x["v"][:, 40 + 50, 1, 3] = float("nan")
    x["k"][:, 40 + 51, 1, 5] = float("inf")
    on, Sn = kda.hd_chunk_fwd(*args, S0=x["S0"], cu_seqlens=cu)
    rn = kda.hd_chunk_bwd(*args, x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=cu)
    assert bool(on[0, 90:150, 1].isnan().any()) and bool(Sn[1, 1].isnan().any())
    on[0, 40 + 32:150, 1] = o[0, 40 + 32:150, 1]
    Sn[1, 1] = S[1, 1]
    assert torch.equal(on, o) and torch.equal(Sn, S)
    for n in ("dq", "dk", "dv", "dg"):
        rn[n][0, 40:150, 1] = r[n][0, 40:150, 1]
        assert torch.equal(rn[n], r[n]), n
    rn["dS0"][1, 1] = r["dS0"][1, 1]
    assert torch.equal(rn["dS0"], r["dS0"])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", [[0, 0, 1, 64, 64, 191, 400], [3, 700, 700, 1180], [0, 1180], [1180, 1180], [0, 0]])
def test_hd_packed(io, cu):
    """Empty sequences, one token, borders inside a chunk, segments; rows outside the sequences stay as they were and
    are not read."""
    T, N = 1200, len(cu) - 1
    x = hd_inputs(1, T, 4, 2, 32, 64, io, 21, N=N)
    out = torch.ones(T, dtype=torch.bool)
    out[cu[0]:cu[-1]] = False
    for n in ("q", "k", "v", "do", "g"):
        x[n][:, out.cuda()] = float("nan")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=c, out=o)
    assert bool((o[:, out.cuda()] == 7.0).all())
    check_fwd(x, o, S, cu=c.cpu())
    res = {n: torch.full_like(x[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c, out=res)
    for n in res:
        assert r[n] is res[n] and bool((r[n][:, out.cuda()] == 7.0).all()), n
    check_bwd(x, r, cu=c.cpu())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_hd_one_long_sequence_among_short_ones(io):
    """Of one packed batch some sequences have many segments, some few, some one."""
    cu = torch.tensor([0, 700, 7900, 7901, 8100, 8990], dtype=torch.int32, device="cuda")
    x = hd_inputs(1, 9000, 1, 1, 32, 32, io, 33, N=5)
    for n in ("q", "k", "v", "do", "g"):
        x[n][:, 8990:] = 0.0
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=cu, out=torch.zeros_like(x["v"]))
    check_fwd(x, o, S, cu=cu.cpu())
    res = {n: torch.zeros_like(x[m]) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=cu, out=res)
    check_bwd(x, r, cu=cu.cpu())


def test_hd_many_packed_sequences():
    """More sequences than the table kernel takes at a time, most of them empty or of one token."""
    N, T = 2500, 3000
    gen = torch.Generator().manual_seed(3)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, 2, (N - 1,), generator=gen).cumsum(0),
                    torch.tensor([T])])
    x = hd_inputs(1, T, 1, 1, 32, 32, "bf16", 31, N=N)
    c = cu.to(torch.int32).cuda()
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=c)
    check_fwd(x, o, S, cu=c.cpu())
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c)
    check_bwd(x, r, cu=c.cpu())


def test_hd_corrupt_cu_seqlens_stay_in_bounds():
    """Entries out of range or falling are clamped and made non-decreasing, as the oracle reads them."""
    x = hd_inputs(1, 300, 2, 2, 32, 32, "bf16", 41, N=5)
    c = torch.tensor([-5, 100, 40, 2 ** 31 - 1, 7, 250], dtype=torch.int32, device="cuda")
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=c)
    check_fwd(x, o, S, cu=c.cpu())
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c)
    check_bwd(x, r, cu=c.cpu())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_hd_strong_decays_and_resets(io):
    """Tokens that clear the state (-inf, and beyond fp32's exponent) between mild ones: exactly nothing passes them,
    and the mild ones keep their precision. No decay at all (g = 0) beside it."""
    x = hd_inputs(1, 200, 3, 3, 64, 32, io, 51)
    g = x["g"]
    g[:, 10::37, 0] = float("-inf")
    g[:, 5::20, 1] = -1000.0
    g[:, 100:130, 1] = -30.0
    g[:, :, 2] = 0.0
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], g, S0=x["S0"])
    check_fwd(x, o, S)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], g, x["do"], S0=x["S0"], dS_final=x["dS"])
    # the oracle's dg of a clearing token is exactly 0, and so is e^g times anything here
    ref = ol.hd_backward(x["q"], x["k"], x["v"], g, x["do"], x["S0"], x["dS"])
    assert bool((ref["dg"][:, 10::37, 0] == 0).all())
    check_bwd(x, r)


def test_hd_empty():
    x = hd_inputs(2, 0, 2, 1, 32, 32, "fp32", 61)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    assert o.shape == (2, 0, 2, 32) and torch.equal(S, x["S0"])
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], dS_final=x["dS"])
    assert torch.equal(r["dS0"], x["dS"]) and r["dg"].shape == (2, 0, 2)
    x = hd_inputs(1, 3, 2, 1, 32, 32, "fp32", 62)
    assert bool((kda.hd_chunk_fwd(x["q"][:, :0], x["k"][:, :0], x["v"][:, :0], x["g"][:, :0])[1] == 0).all())


def test_hd_is_deterministic_whatever_the_workspace_held():
    x = hd_inputs(1, 900, 2, 1, 128, 64, "bf16", 71)
    args = (x["q"], x["k"], x["v"], x["g"])
    wf = torch.empty(kda.hd_workspace_bytes(1, 900, 2, 128, 64, 1, Hk=1), dtype=torch.uint8, device="cuda")
    wb = torch.empty(kda.hd_bwd_workspace_bytes(1, 900, 2, 128, 64, 1, Hk=1), dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0, 255):
        wf.fill_(fill), wb.fill_(fill)
        o, S = kda.hd_chunk_fwd(*args, S0=x["S0"], workspace=wf)
        r = kda.hd_chunk_bwd(*args, x["do"], S0=x["S0"], dS_final=x["dS"], workspace=wb)
        got = {"o": o, "S": S, **r}
        if first is not None:
            for n in got:
                assert torch.equal(got[n], first[n]), n
        first = got


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,Hk,K,V,decay", [(1, 1, 1, 32, 32, "token"), (3, 6, 2, 128, 64, "head"),
                                              (7, 5, 5, 64, 128, "token"), (2, 4, 1, 32, 128, "head"),
                                              (5, 3, 1, 128, 32, "token"), (130, 8, 8, 128, 128, "token")])
def test_hd_decode(N, H, Hk, K, V, decay, io):
    dt = DT[io]
    q, k, v = rnd((N, Hk, K), 1, dt), rnd((N, Hk, K), 2, dt, K ** -0.5), rnd((N, H, V), 3, dt)
    g = -(rnd((N, H) if decay == "token" else (H,), 4) - 2.0).exp()
    g = g.to(dt) if decay == "token" else g
    S = rnd((N, H, K, V), 5)
    if decay == "token":
        g[0, 0] = float("-inf")
    ro, rS = ol.hd_step(q, k, v, g, S, 0.5)
    ao, aS = ol.hd_step(q.abs(), k.abs(), v.abs(), g, S.abs(), 0.5)
    o = kda.hd_decode_step(q, k, v, g, S, scale=0.5)
    close("S", S, rS, 8 * U * aS)  # the decay's exponent and exponential, two products, a sum
    close("o", o, ro, half_step(dt) * ro.abs() + (K + 16) * U * ao)


def test_hd_prefill_then_decode_is_the_whole_sequence():
    """A prompt in chunk form and the rest token by token give what one call over all of it gives."""
    x = hd_inputs(2, 150, 4, 2, 64, 64, "fp32", 81)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    P = 131
    head, Sp = kda.hd_chunk_fwd(*[x[n][:, :P].contiguous() for n in ("q", "k", "v", "g")], S0=x["S0"])
    outs = [head]
    for t in range(P, 150):
        outs.append(kda.hd_decode_step(*[x[n][:, t].contiguous() for n in ("q", "k", "v", "g")], Sp)[:, None])
    check_fwd(x, torch.cat(outs, 1), Sp)
    check_fwd(x, o, S)


def test_hd_long_offsets():
    """Elements past 2^31: the last packed sequences of a batch equal the same sequences alone. (Values are drawn on
    the device: 2^31 of them.)"""
    H, K = 96, 128
    T = (1 << 31) // (H * K) + 5000
    gen = torch.Generator(device="cuda").manual_seed(5)
    big = [torch.empty((1, T, H, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3)]
    g = -torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    cu = torch.tensor([0, T - 4096, T - 77, T], dtype=torch.int32, device="cuda")
    o, S = kda.hd_chunk_fwd(*big, g, cu_seqlens=cu, scale=0.1)
    for n, (a, b) in enumerate([(T - 4096, T - 77), (T - 77, T)]):
        o1, S1 = kda.hd_chunk_fwd(*[t[:, a:b].contiguous() for t in big], g[:, a:b].contiguous(), scale=0.1)
        # the same chunks from the same starts; only the segments' borders differ: two bf16 results of one value
        d = (o[:, a:b].float() - o1.float()).abs()
        assert float((d / (o1.float().abs() + o1.float().abs().mean())).max()) < 2.0 ** -6
        d = (S[n + 1] - S1[0]).abs()
        assert float(d.max()) < 1e-5 * float(S1.abs().max())


def test_hd_gradients_at_long_offsets():
    """The same for the gradients: they equal those of the last sequences alone."""
    H, K = 96, 128
    T = (1 << 31) // (H * K) + 5000
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v, do = [torch.empty((1, T, H, K), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4)]
    g = -torch.rand((1, T, H), device="cuda", generator=gen).to(torch.bfloat16)
    cu = torch.tensor([0, T - 4096, T - 77, T], dtype=torch.int32, device="cuda")
    r = kda.hd_chunk_bwd(q, k, v, g, do, cu_seqlens=cu, scale=0.1)
    for n, (a, b) in enumerate([(T - 4096, T - 77), (T - 77, T)]):
        r1 = kda.hd_chunk_bwd(*[t[:, a:b].contiguous() for t in (q, k, v, g, do)], scale=0.1)
        for name in ("dq", "dk", "dv"):
            x, y = r[name][:, a:b].float(), r1[name].float()
            assert float(((x - y).abs() / (y.abs() + y.abs().mean())).max()) < 2.0 ** -6, name
        d = (r["dS0"][n + 1] - r1["dS0"][0]).abs()
        assert float(d.max()) < 1e-5 * float(r1["dS0"].abs().max())


def test_hd_refusals():
    x = hd_inputs(1, 8, 4, 2, 32, 32, "bf16", 91)
    q, k, v, g = (x[n] for n in ("q", "k", "v", "g"))
    with pytest.raises(ValueError):
        kda.hd_chunk_fwd(q[:, ::2], k, v, g)
    with pytest.raises(ValueError, match="contiguous"):
        kda.hd_chunk_fwd(q, k, torch.empty(1, 8, 32, 4, device="cuda", dtype=torch.bfloat16).transpose(2, 3), g)
    with pytest.raises(TypeError):
        kda.hd_chunk_fwd(q, k, v, g.float())
    with pytest.raises(TypeError):
        kda.hd_chunk_fwd(q, k, v, g[0, 0])  # a constant per head is fp32
    with pytest.raises(ValueError):
        kda.hd_chunk_fwd(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous())
    with pytest.raises(ValueError):
        kda.hd_chunk_bwd(q, k, v, g[0, 0].float(), x["do"], out={"dg": g})
    with pytest.raises(kda.KDAError):
        kda.hd_chunk_fwd(*[torch.zeros(1, 8, 4, 48, device="cuda") for _ in range(3)], torch.zeros(1, 8, 4, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.hd_chunk_fwd(q, k, v, g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    many = [torch.zeros(1, 1, 1 << 16, 32, device="cuda") for _ in range(3)]
    with pytest.raises(kda.KDAError):
        kda.hd_chunk_fwd(*many, torch.zeros(1, 1, 1 << 16, device="cuda"))
    off = torch.zeros(q.numel() + 1, device="cuda", dtype=q.dtype)[1:].view(q.shape)  # 2 bytes behind a 16-byte border
    with pytest.raises(kda.KDAError):
        kda.hd_chunk_fwd(off, k, v, g)
    with pytest.raises(kda.KDAError):
        kda.rotary(off, kda.rotary_freqs(32))
    with pytest.raises(kda.KDAError):
        kda.layer_norm_fwd(off)
    S = torch.zeros(8, 4, 32, 32, device="cuda")
    with pytest.raises(ValueError):
        kda.hd_decode_step(q[0], k[0], v[0], g[0], S[:7])
    with pytest.raises(kda.KDAError):
        kda.hd_decode_step(q[0], k[0], v[0], g[0], S, out=v[0])  # the result may not be an input


# ------------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lead,H,Hk,D,R", [((3, 17), 4, 2, 128, 128), ((5,), 1, 1, 64, 32), ((1, 1), 3, 0, 2, 2),
                                           ((2, 9), 5, 1, 80, 40), ((33,), 2, 2, 96, 22), ((4,), 7, 3, 257, 130),
                                           ((2, 3), 2, 1, 512, 510), ((70,), 96, 8, 128, 64)])
def test_rotary(lead, H, Hk, D, R, layout, io):
    dt = DT[io]
    q, k = rnd((*lead, H, D), 1, dt), rnd((*lead, Hk, D), 2, dt) if Hk else None
    f = kda.rotary_freqs(R)
    for positions in (None, "far"):
        if positions is None:
            pos, given = torch.arange(lead[-1]).expand(lead), None
        else:
            given = torch.randint(-(2 ** 31), 2 ** 31 - 1, lead, generator=torch.Generator().manual_seed(3))
            given = given.to(torch.int32).cuda()
            pos = given
        for inverse, scale in ((False, 1.0), (True, 1.25)):
            got = kda.rotary(q, f, k=k, positions=given, layout=layout, inverse=inverse, scale=scale)
            for x, y in zip((q, k), got if Hk else (got,)):
                ref = ol.rotate(x, f, pos, layout, inverse, scale)
                # sine and cosine: position * 2^-53 of the fp64 frequency (2^31: 2^-22 radians), the reduced angle, the
                # series and the products: together at most 2^-20 of the pair's size; the oracle's own angle is as far
                # off (2^-22) at the farthest positions
                pair = ol.rotate(x.abs(), torch.zeros_like(f), torch.zeros(lead), layout, False, scale)
                first, second = ((slice(0, R // 2), slice(R // 2, R)) if layout == "half"
                                 else (slice(0, R, 2), slice(1, R, 2)))
                size = torch.zeros_like(ref)
                size[..., first] = size[..., second] = pair[..., first] + pair[..., second]
                close(layout, y, ref, half_step(dt) * ref.abs() + 2.0 ** -20 * size)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_in_place_and_back(layout):
    q, k = rnd((2, 50, 4, 64), 1), rnd((2, 50, 2, 64), 2)
    f = kda.rotary_freqs(48)
    want = kda.rotary(q, f, k=k, layout=layout)
    a, b = q.clone(), k.clone()
    got = kda.rotary(a, f, k=b, layout=layout, out=a, k_out=b)
    assert got[0] is a and got[1] is b and torch.equal(a, want[0]) and torch.equal(b, want[1])
    kda.rotary(a, f, k=b, layout=layout, inverse=True, out=a, k_out=b)
    # two rotations of 2^-21 each on pairs of size at most 2 max|x|
    assert float((a - q).abs().max()) <= 2.0 ** -18 * float(q.abs().max())
    assert torch.equal(a[..., 48:], q[..., 48:])


def test_rotary_rejects():
    q, f = rnd((2, 5, 4, 64), 1), kda.rotary_freqs(32)
    with pytest.raises(TypeError):
        kda.rotary(q, f.float())
    with pytest.raises(ValueError):
        kda.rotary(q, f, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        kda.rotary(q, f, positions=torch.zeros(2, 5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        kda.rotary(q, f, layout="quarter")
    with pytest.raises(ValueError):
        kda.rotary(q, f, k=rnd((2, 5, 4, 32), 1))
    with pytest.raises(ValueError):
        kda.rotary(q.transpose(1, 2), f)
    with pytest.raises(kda.KDAError):
        kda.rotary(q, kda.rotary_freqs(66))
    with pytest.raises(kda.KDAError):
        kda.rotary(rnd((1, 1, 1, 600), 1), f)
    assert kda.rotary(q[:0], f).shape == (0, 5, 4, 64)


# ------------------------------------------------------------------------------- layer norm
def norm_inputs(shape, wdim, io, gate, seed):
    dt = DT[io]
    w = {0: None, 1: (shape[-1],), 2: shape[-2:]}[wdim]
    return dict(x=rnd(shape, seed, dt) + 0.5, w=None if w is None else 1 + rnd(w, seed + 1, std=0.3),
                b=None if w is None else rnd(w, seed + 2, std=0.3), z=rnd(shape, seed + 3, dt, 2.0) if gate else None,
                dy=rnd(shape, seed + 4, dt))


NORMS = [((1, 1), 1), ((7, 3), 1), ((5, 16), 0), ((33, 64), 1), ((9, 100), 1), ((3, 5, 128), 2), ((11, 6, 96), 2),
         ((40, 257), 1), ((6, 512), 1), ((4, 1000), 1), ((3, 2049), 1), ((5, 4096), 1), ((2, 7, 700), 2), ((3, 5001), 1),
         ((2, 8192), 1), ((2, 16384), 1), ((3, 9999), 1), ((300, 3, 24), 2), ((1500, 128), 1),
         # more rows than the backward's grid takes at a time: groups that divide a workgroup's rows and that do not
         ((20000, 17), 1), ((9000, 4, 40), 2), ((9000, 3, 128), 2), ((700, 64, 32), 2), ((5000, 2, 300), 2),
         ((1030, 5, 300), 2), ((1100, 2500), 1), ((650, 5001), 1), ((520, 8200), 1), ((515, 9001), 1),
         ((5000, 200), 1), ((4300, 3, 136), 2), ((2000, 513), 1), ((1100, 2, 1024), 2), ((700, 3, 640), 2)]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape,wdim", NORMS)
def test_layer_norm(shape, wdim, gate, center, io):
    dt = DT[io]
    i = norm_inputs(shape, wdim, io, gate, 7)
    x, w, b, z, dy = (i[n] for n in ("x", "w", "b", "z", "dy"))
    kw = dict(weight=w, bias=b, o_gate=z, eps=1e-4, center=center)
    y = kda.layer_norm_fwd(x, **kw)
    ref = ol.norm_forward(x, w, b, z, 1e-4, center)
    # Statistics: sums of C values over at most 16 a thread and 10 halvings, twice, and the handful of operations on
    # each value: under 64 roundings, of (|x| + mean |x|) r where centered, relative to |n| through r.
    n = 64 * U
    xd, C = x.cpu().double(), shape[-1]
    xc = xd - xd.mean(-1, keepdim=True) if center else xd
    r = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-4)
    size = ((xd.abs() + xd.abs().mean(-1, keepdim=True)) * r)  # |n| and what its error is made of
    wd = w.cpu().double().abs() if w is not None else 1.0
    bd = b.cpu().double().abs() if b is not None else 0.0
    a = torch.sigmoid(z.cpu().double()) if gate else 1.0
    # n's error: of its own terms, and through r of the other terms of its row
    nerr = n * size * (1 + size.mean(-1, keepdim=True))
    close("y", y, ref, half_step(dt) * ref.abs() + (nerr * wd + n * (size * wd + bd)) * a)

    res = kda.layer_norm_bwd(dy, x, **kw)
    rb = ol.norm_backward(dy, x, w, b, z, 1e-4, center)
    assert set(res) == set(rb)
    dyd = dy.cpu().double().abs() * a
    d = dyd * wd
    m1, m2 = (d * size).mean(-1, keepdim=True), d.mean(-1, keepdim=True)
    derr = r * (n * (d + size * m1 + m2) + nerr * m1 + size * (d * nerr).mean(-1, keepdim=True)) \
        + r * (d + size * m1 + m2) * n * (1 + size.mean(-1, keepdim=True))
    close("dx", res["dx"], rb["dx"], half_step(dt) * rb["dx"].abs() + derr)
    if gate:
        # a (1 - a): the difference is off by a step of 1, whatever is left of it
        full = dy.cpu().double().abs() * (size * wd + bd)
        close("do_gate", res["do_gate"], rb["do_gate"],
              half_step(dt) * rb["do_gate"].abs() + dy.cpu().double().abs() * nerr * wd * a * (1 - a) + 8 * n * full * a)
    rows = xd.numel() // max(1, w.numel() if w is not None else 1)
    for name, p, e, err in (("dweight", w, dyd * size, dyd * nerr), ("dbias", b, dyd, 0 * dyd)):
        if p is not None:
            # a thread's rows one after the other, then the slots' sums: fewer roundings than rows + 64
            tol = ((rows + 64) * U * e + err + n * e).reshape(-1, *p.shape).sum(0)
            close(name, res[name], rb[name], tol)


def test_layer_norm_special_rows():
    """Constant and zero rows, rows with a large mean, rows with NaN or infinities: they spoil themselves alone."""
    x = rnd((6, 64), 1)
    x[0] = 0.0
    x[1] = 3.0
    x[2] += 1000.0
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    dy = rnd((6, 64), 2)
    y = kda.layer_norm_fwd(x)
    assert bool((y[0] == 0).all()) and bool((y[1] == 0).all())
    assert bool(y[3].isnan().all()) and bool(y[4].isnan().all())
    ref = ol.norm_forward(x, None, None, None)
    # mean 1000 in fp32: the centered values are off by 64 roundings of it
    assert float((y[2].cpu().double() - ref[2]).abs().max()) < 64 * U * 1000 * 4
    assert float((y[5].cpu().double() - ref[5]).abs().max()) < 1e-5
    r = kda.layer_norm_bwd(dy, x)
    assert bool(r["dx"][[0, 1, 2, 5]].isfinite().all()) and bool(r["dx"][3].isnan().all())


def test_layer_norm_rejects_and_empty():
    x = rnd((4, 3, 32), 1)
    w = torch.ones(32, device="cuda")
    for kw in (dict(weight=w[:31]), dict(weight=w.double()), dict(bias=torch.ones(4, 32, device="cuda")),
               dict(weight=w, bias=torch.ones(3, 32, device="cuda")), dict(o_gate=x[0]), dict(o_gate=x.bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            kda.layer_norm_fwd(x, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        kda.layer_norm_fwd(x.transpose(0, 1), weight=w)
    with pytest.raises(kda.KDAError):
        kda.layer_norm_fwd(x, eps=0.0)
    with pytest.raises(kda.KDAError):
        kda.layer_norm_fwd(x, out=x)
    with pytest.raises(kda.KDAError):
        kda.layer_norm_fwd(rnd((1, 16385), 1))
    with pytest.raises(ValueError):
        kda.layer_norm_bwd(x, x, out={"dweight": w})
    e = torch.empty(0, 3, 32, device="cuda")
    assert kda.layer_norm_fwd(e, weight=w).shape == e.shape
    r = kda.layer_norm_bwd(e, e, weight=w, bias=w)
    assert bool((r["dweight"] == 0).all()) and bool((r["dbias"] == 0).all())


def test_long_rows_of_norm_and_rotary():
    """Elements past 2^31: the last rows equal the same rows alone."""
    n = (1 << 31) // 4096 + 300
    x = torch.empty((n, 32, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = 1 + rnd((32, 128), 2, std=0.1)
    assert torch.equal(kda.layer_norm_fwd(x, weight=w)[-200:], kda.layer_norm_fwd(x[-200:].contiguous(), weight=w))
    r = kda.layer_norm_bwd(x, x, weight=w)
    assert torch.equal(r["dx"][-200:], kda.layer_norm_bwd(x[-200:].contiguous(), x[-200:].contiguous(), weight=w)["dx"])
    f = kda.rotary_freqs(128)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    y = kda.rotary(x, f, positions=pos)
    assert torch.equal(y[-200:], kda.rotary(x[-200:].contiguous(), f, positions=pos[-200:].contiguous()))


# ------------------------------------------------------------------------------- streams and graphs
def _layer_calls(io="bf16"):
    x = hd_inputs(1, 700, 2, 1, 64, 64, io, 5, N=3)
    cu = torch.tensor([0, 17, 17, 690], dtype=torch.int32, device="cuda")
    f = kda.rotary_freqs(64)
    w, z = 1 + rnd((2, 64), 1, std=0.2), rnd((1, 700, 2, 64), 2, DT[io])
    S = rnd((700, 2, 64, 64), 3)

    def calls():
        q, k = kda.rotary(x["q"], f, k=x["k"])
        o, Sf = kda.hd_chunk_fwd(q, k, x["v"], x["g"], S0=x["S0"], cu_seqlens=cu, out=torch.zeros_like(x["v"]))
        y = kda.layer_norm_fwd(o, weight=w, o_gate=z)
        r = kda.layer_norm_bwd(x["do"], o, weight=w, o_gate=z)
        res = {n: torch.zeros_like(x[m]) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
        b = kda.hd_chunk_bwd(q, k, x["v"], x["g"], r["dx"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=cu, out=res)
        dq, dk = kda.rotary(b["dq"], f, k=b["dk"], inverse=True)
        St = S.clone()
        od = kda.hd_decode_step(q[0], k[0], x["v"][0], x["g"][0], St)
        return [o, Sf, y, *r.values(), *b.values(), dq, dk, St, od]

    return x, calls


def test_on_another_stream():
    _, calls = _layer_calls()
    want = calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = calls()
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two sequences of calls in flight together, each with its own workspaces."""
    a, b = _layer_calls("bf16")[1], _layer_calls("fp32")[1]
    wa, wb = a(), b()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            ga = a()
        with torch.cuda.stream(t):
            gb = b()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga, wa)) and all(torch.equal(x, y) for x, y in zip(gb, wb))


def test_captured_and_replayed():
    """The whole run in a graph: every replay, on new inputs and with eager work between, equals the eager calls."""
    x, calls = _layer_calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for i in range(4):
        for n in ("q", "k", "v", "do"):
            x[n].copy_(rnd(x[n].shape, 100 + i, x[n].dtype, 0.5))
        x["g"].copy_(-rnd(x["g"].shape, 200 + i).abs().to(x["g"].dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = calls()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


# ------------------------------------------------------------------------------- a layer of them together
def test_layer_forward_gradients_and_tokens():
    """norm -> projections -> rotary -> linear attention -> head norm with gate -> projection: the gradients of the whole
    against fp64 autograd of the definitions, and prompt + tokens against the whole sequence, in fp32.

    Bound: every step is within about 2^-17 of its terms' sizes (some hundred fp32 roundings) and the chain has seven
    steps each way, whose sizes are near those of the results (unit-scale activations and projections): 1e-4 of the
    largest entry."""
    B, T, E, H, Hk, K = 2, 70, 96, 4, 2, 32
    P = {n: rnd(s, i, std=E ** -0.5) for i, (n, s) in enumerate(dict(q=(E, Hk * K), k=(E, Hk * K), v=(E, H * K), z=(E, H * K),
                                                                    g=(E, H), o=(H * K, E)).items())}
    x, dy = rnd((B, T, E), 11), rnd((B, T, E), 12)
    w1, b1, w2 = 1 + rnd((E,), 13, std=0.1), rnd((E,), 14, std=0.1), 1 + rnd((H, K), 15, std=0.1)
    f = kda.rotary_freqs(K)

    def gate(u):  # log-decay of a pre-activation
        return -torch.nn.functional.softplus(u - 2.0)

    # --- the package's operators, forward and backward
    h = kda.layer_norm_fwd(x, weight=w1, bias=b1)
    proj = {n: (h @ P[n]).reshape(B, T, -1, K if n != "g" else 1) for n in "qkvzg"}
    u = proj["g"][..., 0].contiguous()
    q, k = kda.rotary(proj["q"], f, k=proj["k"])
    o, _ = kda.hd_chunk_fwd(q, k, proj["v"], gate(u), scale=K ** -0.5)
    m = kda.layer_norm_fwd(o, weight=w2, o_gate=proj["z"], center=False)
    y = m.reshape(B, T, -1) @ P["o"]
    dm = (dy @ P["o"].T).reshape(m.shape)
    n2 = kda.layer_norm_bwd(dm, o, weight=w2, o_gate=proj["z"], center=False)
    hb = kda.hd_chunk_bwd(q, k, proj["v"], gate(u), n2["dx"], scale=K ** -0.5)
    dq, dk = kda.rotary(hb["dq"], f, k=hb["dk"], inverse=True)
    du = hb["dg"] * -torch.sigmoid(u - 2.0)
    dh = sum(d.reshape(B, T, -1) @ P[n].T for n, d in (("q", dq), ("k", dk), ("v", hb["dv"]), ("z", n2["do_gate"]), ("g", du)))
    n1 = kda.layer_norm_bwd(dh, x, weight=w1, bias=b1)
    got = {"y": y, "dx": n1["dx"], "dw1": n1["dweight"], "db1": n1["dbias"], "dw2": n2["dweight"],
           "dPq": h.reshape(-1, E).T @ dq.reshape(B * T, -1), "dPg": h.reshape(-1, E).T @ du.reshape(B * T, -1)}

    # --- fp64 autograd of the definitions
    X, W1, B1, W2 = (ol.f64(t).requires_grad_() for t in (x, w1, b1, w2))
    Q = {n: ol.f64(t).requires_grad_() for n, t in P.items()}
    hh = torch.nn.functional.layer_norm(X, (E,), W1, B1, 1e-5)
    p = {n: (hh @ Q[n]).reshape(B, T, -1, K if n != "g" else 1) for n in "qkvzg"}
    angle = torch.arange(T, dtype=torch.float64)[:, None, None] * ol.f64(f)
    c, s = torch.cos(angle), torch.sin(angle)
    turn = lambda t: torch.cat([t[..., :K // 2] * c - t[..., K // 2:] * s, t[..., :K // 2] * s + t[..., K // 2:] * c], -1)  # noqa: E731
    qq, kk = (turn(p[n]).repeat_interleave(H // Hk, 2) for n in "qk")
    a = torch.exp(gate(p["g"][..., 0]))
    S, outs = torch.zeros(B, H, K, K, dtype=torch.float64), []
    for t in range(T):
        S = a[:, t, :, None, None] * S + kk[:, t, :, :, None] * p["v"][:, t, :, None, :]
        outs.append(K ** -0.5 * (qq[:, t, :, :, None] * S).sum(2))
    oo = torch.stack(outs, 1)
    mm = oo / torch.sqrt((oo * oo).mean(-1, keepdim=True) + 1e-5) * W2 * torch.sigmoid(p["z"])
    yy = mm.reshape(B, T, -1) @ Q["o"]
    (yy * ol.f64(dy)).sum().backward()
    want = {"y": yy.detach(), "dx": X.grad, "dw1": W1.grad, "db1": B1.grad, "dw2": W2.grad, "dPq": Q["q"].grad,
            "dPg": Q["g"].grad}
    for n in want:
        assert float((got[n].cpu().double() - want[n]).abs().max()) <= 1e-4 * float(want[n].abs().max()), n

    # --- the last tokens one by one
    n = 60
    part = lambda t: t[:, :n].contiguous()  # noqa: E731
    _, S = kda.hd_chunk_fwd(part(q), part(k), part(proj["v"]), part(gate(u)), scale=K ** -0.5)
    for t in range(n, T):
        h1 = kda.layer_norm_fwd(x[:, t].contiguous(), weight=w1, bias=b1)
        pr = {c: (h1 @ P[c]).reshape(B, -1, K if c != "g" else 1) for c in "qkvzg"}
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        q1, k1 = kda.rotary(pr["q"], f, k=pr["k"], positions=pos)
        o1 = kda.hd_decode_step(q1, k1, pr["v"], gate(pr["g"][..., 0]).contiguous(), S, scale=K ** -0.5)
        m1 = kda.layer_norm_fwd(o1, weight=w2, o_gate=pr["z"], center=False)
        y1 = m1.reshape(B, -1) @ P["o"]
        assert float((y1.cpu().double() - want["y"][:, t]).abs().max()) <= 1e-4 * float(want["y"].abs().max())
