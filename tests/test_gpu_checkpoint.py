"""GPU tests of the rotary positions with several axes and of the checkpoints in 8 bits against their fp64 definitions
(oracle.layers), and of a layer that uses the operators together.

Tolerances: half a step of the result's type relative to the value; a rotation adds the error of fp32 sines, products and a
sum, 8 roundings of 2^-24 of |x1| + |x2|. A checkpoint's codes are whole numbers and have to be equal."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import delta as od
from oracle import layers as ol
from tests.test_gpu_layers import DT, U, close, half_step, rnd

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ rotary axes
def check_axes(x, y, freqs, axes, pos, layout, inverse, scale):
    ref = ol.rotate_axes(x, freqs, axes, pos, layout, inverse, scale)
    P = freqs.numel()
    mag = ref.abs()
    one, two = (slice(0, P), slice(P, 2 * P)) if layout == "half" else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
    a = ol.f64(x).abs()
    for part in (one, two):
        mag[..., part] = abs(scale) * (a[..., one] + a[..., two])
    close("rotated", y, ref, half_step(x.dtype) * ref.abs() + 8 * U * mag)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lead,H,Hk,D,sections,order", [
    ((1,), 1, 1, 32, [16], "runs"), ((33,), 5, 1, 64, [10, 11, 11], "turns"), ((2, 17), 4, 2, 128, [16, 24, 24], "runs"),
    ((3, 50), 3, 3, 80, [20, 20], "runs"), ((7,), 2, 1, 96, [1, 2, 3], "turns"), ((2, 9), 8, 8, 256, [5, 60, 60], "turns"),
    ((70,), 6, 2, 36, [3, 4, 4], "runs"), ((5,), 1, 1, 6, [1, 1, 1], "runs")])
def test_axes(lead, H, Hk, D, sections, order, layout, io):
    dt, n = DT[io], sum(sections)
    q, k = rnd((*lead, H, D), 1, dt), rnd((*lead, Hk, D), 2, dt)
    freqs, axes = kda.rotary_freqs(2 * n), kda.rotary_sections(sections, order)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (len(sections), *lead), generator=torch.Generator().manual_seed(3),
                        dtype=torch.int64).to(torch.int32).cuda()
    for inverse, scale in ((False, 1.0), (True, 0.7)):
        y, z = kda.rotary_axes(q, freqs, axes, pos, k=k, layout=layout, inverse=inverse, scale=scale)
        check_axes(q, y, freqs, axes, pos, layout, inverse, scale)
        check_axes(k, z, freqs, axes, pos, layout, inverse, scale)
    alone = kda.rotary_axes(q, freqs, axes, pos, layout=layout, inverse=True, scale=0.7)
    assert torch.equal(alone, y)
    a, b = q.clone(), k.clone()  # in place
    kda.rotary_axes(a, freqs, axes, pos, k=b, layout=layout, inverse=True, scale=0.7, out=a, k_out=b)
    assert torch.equal(a, y) and torch.equal(b, z)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_equal_axes_are_the_plain_rotation(layout):
    """Every axis at the same position: bit for bit what rotary() gives."""
    q, freqs = rnd((2, 40, 4, 64), 5, torch.bfloat16), kda.rotary_freqs(48)
    pos = torch.arange(80, dtype=torch.int32, device="cuda").reshape(2, 40) * 1000
    axes = kda.rotary_sections([8, 8, 8], "turns")
    got = kda.rotary_axes(q, freqs, axes, pos.expand(3, 2, 40).contiguous(), layout=layout)
    assert torch.equal(got, kda.rotary(q, freqs, positions=pos, layout=layout))


def test_the_inverse_is_the_gradient():
    """<R q, y> = <q, R^T y> for the rotation and its inverse, in fp32: sums of 2 * 1e4 terms of size one, each off by 8
    roundings, independent of each other: 16 * sqrt(1e4) * 2^-24 = 1e-4 with room."""
    q, y = rnd((50, 4, 64), 7), rnd((50, 4, 64), 8)
    freqs, axes = kda.rotary_freqs(64), kda.rotary_sections([12, 10, 10])
    pos = torch.randint(0, 5000, (3, 50), generator=torch.Generator().manual_seed(9)).to(torch.int32).cuda()
    a = (kda.rotary_axes(q, freqs, axes, pos, scale=1.3).double() * y.double()).sum()
    b = (q.double() * kda.rotary_axes(y, freqs, axes, pos, scale=1.3, inverse=True).double()).sum()
    assert abs(float(a - b)) < 1e-3


def test_unknown_axes_and_frequencies_make_their_pairs_nan():
    q, freqs = rnd((6, 2, 32), 11), kda.rotary_freqs(32)
    axes = kda.rotary_sections([8, 8])
    pos = torch.arange(12, dtype=torch.int32, device="cuda").reshape(2, 6)
    clean = kda.rotary_axes(q, freqs, axes, pos)
    axes[3], axes[9], freqs[5] = 2, -1, float("inf")
    y = kda.rotary_axes(q, freqs, axes, pos)
    bad = torch.zeros(32, dtype=torch.bool, device="cuda")
    for j in (3, 9, 5):
        bad[j] = bad[j + 16] = True
    assert bool(y[..., bad].isnan().all()) and torch.equal(y[..., ~bad], clean[..., ~bad])


def test_axes_refusals():
    q, freqs, axes = rnd((6, 2, 32), 13), kda.rotary_freqs(16), kda.rotary_sections([4, 4])
    pos = torch.zeros((2, 6), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        kda.rotary_axes(q, freqs, axes[:7], pos)
    with pytest.raises(TypeError):
        kda.rotary_axes(q, freqs, axes.long(), pos)
    with pytest.raises(ValueError):
        kda.rotary_axes(q, freqs, axes, pos[:, :5])
    with pytest.raises(TypeError):
        kda.rotary_axes(q, freqs, axes, pos.float())
    with pytest.raises(kda.KDAError):
        kda.rotary_axes(q, freqs, axes, torch.zeros((17, 6), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kda.rotary_axes(q, freqs, axes, pos, layout="thirds")
    with pytest.raises(ValueError):
        kda.rotary_axes(q, freqs, axes, pos, k_out=q)


# ------------------------------------------------------------------------------------------ checkpoints
SHAPES = [(1, 1), (3, 7), (5, 32), (9, 64), (4, 100), (6, 128), (7, 129), (2, 3, 96), (11, 300), (2, 5, 4, 128), (1, 4096),
          (300, 513), (17, 1000)]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_save_and_restore(shape, io):
    x = rnd(shape, 21, DT[io])
    x *= torch.exp(2 * rnd((*shape[:-1], 1), 22)).to(DT[io])
    codes, scales = ol.save8(x)
    c = kda.checkpoint8(x)
    assert c.codes.dtype is torch.int8 and c.dtype is DT[io]
    # fp32: 127 x is rounded, a quotient within 2^-22 of a half can go either way
    off = (c.codes.cpu().int() - codes.int()).abs()
    assert int(off.max()) == 0 if io == "bf16" else float((off > 0).float().mean()) < 1e-4 and int(off.max()) <= 1
    close("scales", c.scales, scales, U * scales * 1.01)
    y = kda.restore8(c)
    ref = ol.restore8(c.codes, c.scales)
    close("restored", y, ref, half_step(DT[io]) * ref.abs())
    into = kda.Checkpoint8(torch.full_like(c.codes, 99), torch.full_like(c.scales, -1.0), x.dtype)
    assert kda.checkpoint8(x, out=into) is into and torch.equal(into.codes, c.codes) and torch.equal(into.scales, c.scales)
    z = torch.empty_like(x)
    assert kda.restore8(c, out=z) is z and torch.equal(z, y)
    assert torch.equal(kda.checkpoint8(y).codes, c.codes) or io == "bf16"  # fp32: what was restored is saved unchanged


def test_ties_go_to_the_even_code():
    """Quotients of a half exactly: x = top (m + 1/2) / 127 for a top of 127 steps of 2."""
    x = torch.tensor([254.0, 1.0, 3.0, 5.0, -1.0, -3.0, 127.0, 129.0, -253.0, 0.0]).cuda()
    want = [127, 0, 2, 2, 0, -2, 64, 64, -126, 0]
    for dt in (torch.float32, torch.bfloat16):
        assert kda.checkpoint8(x.to(dt)).codes.tolist() == want


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120])
def test_very_small_and_large_values(size, io):
    x = (rnd((40, 256), 23).clamp(-8, 8) * size).to(DT[io])
    codes, _ = ol.save8(x)
    c = kda.checkpoint8(x)
    assert float((c.codes.cpu() != codes).float().mean()) < (1e-4 if io == "fp32" else 1e-9)
    step = c.scales.double().cpu().repeat_interleave(128, dim=1)
    close("restored", kda.restore8(c), ol.f64(x), (0.5 + 128 * half_step(DT[io])) * step * 1.001)


def test_zeros_infinities_and_nan():
    x = rnd((4, 300), 24)
    x[0, :128] = 0.0
    x[1, 130] = float("inf")
    x[2, 299] = float("nan")
    x[3, 5] = -float("inf")
    clean = rnd((4, 300), 24)
    y, ref = kda.restore8(kda.checkpoint8(x)), kda.restore8(kda.checkpoint8(clean))
    assert bool((y[0, :128] == 0).all())
    for row, a, b in ((1, 128, 256), (2, 256, 300), (3, 0, 128)):
        assert bool(y[row, a:b].isnan().all())
        y[row, a:b] = ref[row, a:b]
    y[0, :128] = ref[0, :128]
    assert torch.equal(y, ref)


def test_empty_checkpoint():
    c = kda.checkpoint8(torch.empty((0, 5), device="cuda"))
    assert c.codes.shape == (0, 5) and c.scales.shape == (0, 1) and kda.restore8(c).shape == (0, 5)


def test_checkpoint_long_offsets():
    """Values past 2^31: the last rows are those of the same rows alone."""
    rows, C = (1 << 31) // 4096 + 9, 4096
    x = torch.empty((rows, C), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    c, tail = kda.checkpoint8(x), kda.checkpoint8(x[-5:].contiguous())
    assert torch.equal(c.codes[-5:], tail.codes) and torch.equal(c.scales[-5:], tail.scales)
    assert torch.equal(kda.restore8(c)[-5:], kda.restore8(tail))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H,C,gate,center,bias", [
    (1, 1, 1, False, True, True), (5, 1, 33, True, True, False), (64, 1, 128, False, False, False), (30, 3, 100, True, True, True),
    (9, 4, 64, True, False, False), (40, 1, 520, False, True, True), (33, 1, 1000, True, True, False),
    (7, 1, 2048, False, True, True), (6, 1, 4100, True, False, True), (5, 1, 9000, False, True, False), (600, 2, 48, True, True, True)])
def test_norm_gradients_from_a_checkpoint(rows, H, C, gate, center, bias, io):
    """Bit for bit those of the values that the checkpoint stands for."""
    dt = DT[io]
    shape, wshape = ((rows, H, C), (H, C)) if H > 1 else ((rows, C), (C,))
    saved = kda.checkpoint8(rnd(shape, 31, dt))
    dy, w = rnd(shape, 32, dt), rnd(wshape, 33)
    b, z = rnd(wshape, 34) if bias else None, rnd(shape, 35, dt) if gate else None
    got = kda.layer_norm_bwd(dy, saved, weight=w, bias=b, o_gate=z, center=center)
    want = kda.layer_norm_bwd(dy, kda.restore8(saved), weight=w, bias=b, o_gate=z, center=center)
    assert set(got) == set(want)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_checkpoint_refusals():
    x = rnd((4, 300), 41, torch.bfloat16)
    c = kda.checkpoint8(x)
    with pytest.raises(TypeError):
        kda.checkpoint8(x.half())
    with pytest.raises(ValueError, match="contiguous"):
        kda.checkpoint8(x.t())
    with pytest.raises(TypeError):
        kda.checkpoint8(x, out=c._replace(dtype=torch.float32))
    with pytest.raises(ValueError):
        kda.checkpoint8(x, out=c._replace(scales=c.scales[:, :2]))
    with pytest.raises(TypeError):
        kda.restore8(c._replace(codes=c.codes.int()))
    with pytest.raises(TypeError):
        kda.layer_norm_bwd(x.float(), c)
    with pytest.raises(ValueError):
        kda.layer_norm_bwd(x[:3], c)
    with pytest.raises(kda.KDAError):  # 1 byte behind a 16-byte border
        kda.restore8(c._replace(codes=torch.empty(1201, dtype=torch.int8, device="cuda")[1:].view(4, 300)))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_recurrences_from_checkpoints(io):
    """The gradients of both recurrences with q, k and v out of checkpoints, or some of them."""
    dt = DT[io]
    q, k, v = rnd((2, 90, 2, 64), 51, dt), rnd((2, 90, 2, 64), 52, dt, 0.125), rnd((2, 90, 4, 32), 53, dt)
    g, beta = (-rnd((2, 90, 4), 54).exp()).to(dt), torch.sigmoid(rnd((2, 90, 4), 55)).to(dt)
    do = rnd((2, 90, 4, 32), 56, dt)
    cq, ck, cv = (kda.checkpoint8(t) for t in (q, k, v))
    rq, rk, rv = (kda.restore8(t) for t in (cq, ck, cv))
    for got, want in ((kda.gd_chunk_bwd(cq, ck, cv, g, beta, do), kda.gd_chunk_bwd(rq, rk, rv, g, beta, do)),
                      (kda.gd_chunk_bwd(q, ck, v, g, beta, do), kda.gd_chunk_bwd(q, rk, v, g, beta, do)),
                      (kda.hd_chunk_bwd(cq, ck, cv, g, do), kda.hd_chunk_bwd(rq, rk, rv, g, do))):
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_a_layer_of_the_operators_together():
    """Norm, gated delta rule with keys of length one, gated norm behind it, and beside it the rotation of an attention's
    q and k by three axes: forward; then backward from inputs kept in 8 bits, against the gradients of the same layer at
    the kept values in fp64 (autograd over the oracle's lines)."""
    B, T, H, K, V, C = 1, 45, 2, 32, 32, 64
    x = rnd((B, T, C), 61)
    saved = kda.checkpoint8(x)
    x = kda.restore8(saved)
    wn = 1.0 + 0.1 * rnd((C,), 62)
    proj = {n: rnd((C, s), 63 + i, std=C ** -0.5) for i, (n, s) in enumerate((("q", H * K), ("k", H * K), ("v", H * V)))}
    g, beta = -rnd((B, T, H), 67).exp(), torch.sigmoid(rnd((B, T, H), 68))
    unit = torch.full((K,), K ** -0.5, device="cuda")
    wo, gate, dy = 1.0 + 0.1 * rnd((H, V), 69), rnd((B, T, H, V), 70), rnd((B, T, H, V), 71)

    # ---- the package
    n = kda.layer_norm_fwd(x, weight=wn, center=False)
    q, k, v = ((n @ proj[m]).reshape(B, T, H, -1) for m in "qkv")
    kn = kda.layer_norm_fwd(k, weight=unit, center=False, eps=1e-6)
    o, S = kda.gd_chunk_fwd(q, kn, v, g, beta, scale=K ** -0.5)
    y = kda.layer_norm_fwd(o, weight=wo, o_gate=gate, center=False)
    out = kda.layer_norm_bwd(dy, o, weight=wo, o_gate=gate, center=False)
    r = kda.gd_chunk_bwd(q, kn, v, g, beta, out["dx"], scale=K ** -0.5)
    dk = kda.layer_norm_bwd(r["dk"], k, weight=unit, center=False, eps=1e-6)["dx"]
    dn = sum(t.reshape(B, T, -1) @ proj[m].t() for t, m in ((r["dq"], "q"), (dk, "k"), (r["dv"], "v")))
    back = kda.layer_norm_bwd(dn, saved, weight=wn, center=False)

    # ---- the same in fp64
    X, WN, WO = (ol.f64(t).requires_grad_() for t in (x, wn, wo))
    P = {m: ol.f64(t) for m, t in proj.items()}
    N = X / torch.sqrt((X * X).mean(-1, keepdim=True) + 1e-5) * WN
    Q, Kr, Vv = ((N @ P[m]).reshape(B, T, H, -1) for m in "qkv")
    Kn = Kr / torch.sqrt((Kr * Kr).mean(-1, keepdim=True) + 1e-6) * ol.f64(unit)
    St, os = torch.zeros(B, H, K, V, dtype=torch.float64), []
    for t in range(T):
        St = torch.exp(ol.f64(g)[:, t])[..., None, None] * St
        z = Vv[:, t] - (Kn[:, t][..., None] * St).sum(2)
        St = St + (ol.f64(beta)[:, t][..., None] * Kn[:, t])[..., None] * z[:, :, None]
        os.append(K ** -0.5 * (Q[:, t][..., None] * St).sum(2))
    O = torch.stack(os, 1)
    Y = O / torch.sqrt((O * O).mean(-1, keepdim=True) + 1e-5) * WO * torch.sigmoid(ol.f64(gate))
    (Y * ol.f64(dy)).sum().backward()

    def near(a, ref):  # fp32 throughout: products of 64 terms and the passes' own errors, some 2^-17 in all
        return float((a.cpu().double() - ref).norm() / ref.norm()) < 2.0 ** -16

    assert near(y, Y.detach()) and near(S, St.detach())
    assert near(back["dx"], X.grad) and near(back["dweight"], WN.grad) and near(out["dweight"], WO.grad)

    # ---- the attention's positions: rotated, and the gradient turned back
    freqs, axes = kda.rotary_freqs(K), kda.rotary_sections([4, 6, 6])
    pos = torch.stack([torch.arange(T) // 9, torch.arange(T) % 9 // 3, torch.arange(T) % 3]).to(torch.int32)[:, None].cuda()
    rq, rk = kda.rotary_axes(q, freqs, axes, pos.contiguous(), k=kn)
    check_axes(q, rq, freqs, axes, pos, "half", False, 1.0)
    back_q = kda.rotary_axes(rq, freqs, axes, pos.contiguous(), inverse=True)
    assert float((back_q - q).abs().max()) < 32 * U * float(q.abs().max())
