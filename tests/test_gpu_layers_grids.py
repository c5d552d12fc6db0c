"""GPU tests of the operators around the recurrence where a grid is smaller than the work (its workgroups walk on) or
larger than one dimension, and of many rows' sums, against the fp64 definitions (oracle.layers) or plain fp64 torch."""
import math

import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import layers as ol
from tests.test_gpu_layers import DT, U, check_bwd, check_fwd, close, half_step, hd_inputs, rnd
from tests.test_gpu_layers import test_layer_norm as check_norm

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- single tokens
# Up to 4096 (sequence, head) pairs take a workgroup each; above that a workgroup walks over pairs, a ragged number of them.
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,Hk,K,V,decay", [(515, 8, 8, 32, 32, "token"), (515, 8, 2, 32, 32, "head"),
                                              (2101, 9, 3, 32, 32, "token"), (2101, 9, 9, 32, 32, "head"),
                                              (1031, 4, 2, 64, 128, "token"), (4099, 1, 1, 128, 32, "token"),
                                              (460, 9, 1, 128, 128, "head")])
def test_decode_walks(N, H, Hk, K, V, decay, io):
    dt = DT[io]
    q, k, v = rnd((N, Hk, K), 1, dt), rnd((N, Hk, K), 2, dt, K ** -0.5), rnd((N, H, V), 3, dt)
    g = -(rnd((N, H) if decay == "token" else (H,), 4) - 2.0).exp()
    g = g.to(dt) if decay == "token" else g
    S = rnd((N, H, K, V), 5)
    ro, rS = ol.hd_step(q, k, v, g, S, 0.5)
    ao, aS = ol.hd_step(q.abs(), k.abs(), v.abs(), g, S.abs(), 0.5)
    o = kda.hd_decode_step(q, k, v, g, S, scale=0.5)
    close("S", S, rS, 8 * U * aS)  # the decay's exponent and exponential, two products, a sum
    close("o", o, ro, half_step(dt) * ro.abs() + (K + 16) * U * ao)


def test_decode_of_more_pairs_than_any_grid():
    """2^23 + 1 pairs (34 GB of states): the grid's own cap. Slice by slice, on the device in fp64."""
    H, K = 3, 32
    N = (2 ** 23 + 1) // H
    assert N * H == 2 ** 23 + 1
    S = torch.empty(N, H, K, K, device="cuda")
    cuts = list(range(0, N, 2 ** 16)) + [N]

    def fill(i, out):
        gen = torch.Generator("cuda").manual_seed(i)
        return out.normal_(generator=gen)

    gen = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.randn(N, H, K, device="cuda", generator=gen) for _ in range(3))
    g = -torch.rand(N, H, device="cuda", generator=gen)
    for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
        fill(i, S[a:b])
    o = kda.hd_decode_step(q, k, v, g, S)
    for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
        S0 = fill(i, torch.empty_like(S[a:b])).double()
        d, kv = g[a:b].double().exp()[..., None, None], k[a:b].double()[..., None] * v[a:b].double()[..., None, :]
        ref = d * S0 + kv
        assert bool(((S[a:b].double() - ref).abs() <= 8 * U * (d * S0.abs() + kv.abs())).all()), i
        qd = q[a:b].double()[..., None]
        err = (o[a:b].double() - (qd * ref).sum(2)).abs()
        assert bool((err <= (K + 17) * U * (qd.abs() * (d * S0.abs() + kv.abs())).sum(2)).all()), i


# ------------------------------------------------------------------------------- many sequences
@pytest.mark.parametrize("packed", [False, True])
def test_more_sequences_than_a_grid_dimension(packed):
    """2^20 + 50 sequences of two tokens (a grid's first dimension has 2^20 workgroups), fp32: both passes against the two
    tokens' formulas and their autograd in fp64."""
    N, K = 2 ** 20 + 50, 32
    gen = torch.Generator("cuda").manual_seed(9)
    shape = (1, 2 * N, 1, K) if packed else (N, 2, 1, K)
    q, k, v, do = (torch.randn(shape, device="cuda", generator=gen) for _ in range(4))
    g = -torch.rand(shape[:3], device="cuda", generator=gen)
    dS = torch.randn(N, 1, K, K, device="cuda", generator=gen)
    cu = torch.arange(0, 2 * N + 1, 2, dtype=torch.int32, device="cuda") if packed else None
    o, S = kda.hd_chunk_fwd(q, k, v, g, cu_seqlens=cu, scale=0.5)
    r = kda.hd_chunk_bwd(q, k, v, g, do, dS_final=dS, cu_seqlens=cu, scale=0.5)

    def definition(q, k, v, g, do, dS):
        """o, S and, of <o, do> + <S, dS>, the gradients."""
        q, k, v, g = (x.double().requires_grad_() for x in (q, k, v, g))
        w = g[:, 1].exp()
        kv = lambda i: k[:, i, :, None] * v[:, i, None, :]  # noqa: E731
        s0 = kv(0)
        s1 = w[:, None, None] * s0 + kv(1)
        o = 0.5 * torch.stack([(q[:, 0, :, None] * s0).sum(1), (q[:, 1, :, None] * s1).sum(1)], 1)
        grads = torch.autograd.grad((o * do.double()).sum() + (s1 * dS.double()).sum(), (q, k, v, g))
        return o.detach(), s1.detach(), dict(zip(("dq", "dk", "dv", "dg"), grads))

    # roundings on a term's way: two dot products of K, the weights, a chunk's two sources, the states' sums
    n = 2 * K + 2 * K + 64 + 16
    flat = lambda x: x.reshape(N, 2, -1)  # noqa: E731
    for a in range(0, N, 2 ** 17):
        b = min(a + 2 ** 17, N)
        part = [flat(x)[a:b] for x in (q, k, v)] + [g.reshape(N, 2)[a:b]] + [flat(do)[a:b], dS[a:b, 0]]
        ro, rS, rg = definition(*part)
        ao, aS, ag = definition(*[x if i == 3 else x.abs() for i, x in enumerate(part)])
        assert bool(((flat(o)[a:b].double() - ro).abs() <= n * U * ao).all())
        assert bool(((S[a:b, 0].double() - rS).abs() <= n * U * aS).all())
        for name in ("dq", "dk", "dv"):
            assert bool(((flat(r[name])[a:b].double() - rg[name]).abs() <= n * U * ag[name]).all()), name
        # dg is summed from the tokens' q.dq less k.dk behind them (their absolute sums bound it) and <S, dS>
        parts = (part[0].abs().double() * ag["dq"]).sum(2) + (part[1].abs().double() * ag["dk"]).sum(2)
        tol = parts.flip(1).cumsum(1).flip(1) + (aS * part[5].abs().double()).sum((1, 2))[:, None]
        assert bool(((r["dg"].reshape(N, 2)[a:b].double() - rg["dg"]).abs() <= n * U * tol).all())


# ------------------------------------------------------------------------------- scales and decays over segments
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("T,H,Hk,K,V,cu", [(1537, 1, 1, 64, 64, None), (2100, 2, 1, 128, 64, None), (9000, 1, 1, 32, 32, None),
                                           (1500, 3, 1, 64, 128, [0, 700, 700, 1400, 1500]),
                                           (9000, 1, 1, 32, 32, [0, 700, 7900, 7901, 9000])])
def test_hd_scales_and_decays_over_segments(T, H, Hk, K, V, cu, decay, io):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    x = hd_inputs(1, T, H, Hk, K, V, io, 800, decay, N=1 if cu is None else len(cu) - 1)
    host = None if cu is None else torch.tensor(cu)
    for scale in (0.3, -1.7):
        o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=c, scale=scale)
        check_fwd(x, o, S, cu=host, scale=scale)
        r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c, scale=scale)
        check_bwd(x, r, cu=host, scale=scale, decay=decay)


# ------------------------------------------------------------------------------- norm rows beyond one grid
# The forward grid has at most 2048 workgroups: rows of 513 channels (two a workgroup) and more take several turns.
WALKS = [((4200, 513), 1), ((2100, 1025), 1), ((2100, 2, 700), 2), ((2100, 4096), 1), ((2100, 5001), 1), ((2060, 9001), 1),
         ((2055, 9008), 1)]


@pytest.mark.parametrize("io,gate,center", [("bf16", True, True), ("fp32", False, False), ("bf16", False, True),
                                            ("fp32", True, False)])
@pytest.mark.parametrize("shape,wdim", WALKS)
def test_layer_norm_walks(shape, wdim, io, gate, center):
    if shape[-1] <= 2048 or (io, gate) in (("bf16", True), ("fp32", False)):  # the oracle's share of the time
        check_norm(shape, wdim, gate, center, io)
    x, z = rnd(shape, 1, DT[io]), rnd(shape, 2, DT[io]) if gate else None
    w, b = 1 + rnd(shape[-wdim:], 3, std=0.2), rnd(shape[-wdim:], 4, std=0.2)
    y = kda.layer_norm_fwd(x, weight=w, bias=b, o_gate=z, center=center)
    # a row's result does not depend on the others: in parts that are one turn each (copies: aligned whatever the width)
    for a in range(0, shape[0], 700):
        part = [None if t is None else t[a:a + 700].clone() for t in (x, z)]
        assert torch.equal(y[a:a + 700], kda.layer_norm_fwd(part[0], weight=w, bias=b, o_gate=part[1], center=center))


# ------------------------------------------------------------------------------- parameter gradients of many rows
MANY = [(20000, 1, 17), (9000, 4, 40), (9000, 3, 128), (700, 64, 32), (5000, 2, 300), (1030, 5, 300), (1100, 1, 2500),
        (650, 1, 5001), (520, 1, 8200), (515, 1, 9001), (5000, 1, 200), (4300, 3, 136), (2000, 1, 513), (1100, 2, 1024),
        (16385, 1, 64), (16384, 1, 64), (511, 7, 64), (513, 1, 4096), (1, 1, 64), (31, 33, 8)]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,G,C", MANY)
def test_layer_norm_parameter_gradients_count_every_row_once(rows, G, C, io):
    """dbias of whole numbers is exact in fp32, whatever the order. dweight, of gradients in a few rows (the last ones, and
    some of every turn), is within a bound that is less than one such row's share."""
    gen = torch.Generator().manual_seed(rows)
    dy = torch.randint(-3, 5, (rows, G, C), generator=gen)
    x = rnd((rows, G, C), 5, DT[io])
    w, b = torch.ones(G, C, device="cuda"), torch.zeros(G, C, device="cuda")
    r = kda.layer_norm_bwd(dy.to(DT[io]).cuda(), x, weight=w, bias=b, eps=1e-4)
    assert torch.equal(r["dbias"].cpu().double(), dy.sum(0).double())

    few = torch.zeros(rows, dtype=torch.bool)
    few[:: max(1, rows // 40)] = True
    few[-40:] = True
    dy *= few[:, None, None]
    r = kda.layer_norm_bwd(dy.to(DT[io]).cuda(), x, weight=w, bias=b, eps=1e-4)
    assert torch.equal(r["dbias"].cpu().double(), dy.sum(0).double())
    # A row slot adds its rows, a workgroup its slots, 16 wavefronts every 16th partial row, one adds these.
    per_wg = 32 if C <= 64 else 16 if C <= 128 else 8 if C <= 256 else 4 if C <= 512 else 2 if C <= 1024 else 1
    step = G // math.gcd(G, per_wg)
    wgs = (min(-(-rows * G // per_wg), 512) + step - 1) // step * step
    depth = -(-rows * G // (wgs * per_wg)) + per_wg + -(-wgs * per_wg // (16 * G)) + 16
    xd = x.cpu().double()
    xc = xd - xd.mean(-1, keepdim=True)
    rs = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-4)
    size = (xd.abs() + xd.abs().mean(-1, keepdim=True)) * rs
    nerr = 64 * U * size * (1 + size.mean(-1, keepdim=True))  # of a normed value: its statistics and operations
    e = dy.abs().double()
    tol = ((depth * U) * (e * (xc * rs).abs()) + e * nerr).sum(0)
    close("dweight", r["dweight"], (dy.double() * xc * rs).sum(0), tol)
    assert float((tol * few.sum() / (e * (xc * rs).abs()).sum(0).clamp(min=1e-9)).min()) < 0.1  # of a row's share
