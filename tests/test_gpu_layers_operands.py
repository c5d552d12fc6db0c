"""GPU tests of the bf16 operands of linear attention with one decay per head, against fp64 (oracle.layers).

Where a computed fp32 value enters a matrix product of bf16 operands it goes in as two parts, hi = bf16(x) and
lo = bf16(x - hi): |x - hi| <= 2^-8 |x|, and lo is off by at most 2^-8 of that, so the pair holds x to 2^-16. A term of
a result passes one such operand (a weighted product, or the state), so the operands cost 2^-16 of the sum of the
terms' absolute values; with one part they would cost up to 2^-8 of it. On top come the fp32 roundings on a term's way
and half a step of the result's type.
"""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import layers as ol
from tests.test_gpu_layers import DT, U, _abs, close, half_step, hd_inputs

pytestmark = pytest.mark.gpu

PAIR = {"bf16": 2.0 ** -16, "fp32": 0.0}


def roundings(T, K, V, group=1):
    """fp32 roundings on a term's way: its dot product over K or V channels, its weight (exponent, exponential, factors:
    16), the sums over a chunk's 32 sources and the state's channels in two parts each, over the chunks before (a product
    and a sum each), over the heads that share a row."""
    return (K + V) + 2 * (32 + max(K, V)) + 2 * (T // 32 + 1) + 16 + group


CASES = [  # B, T, H, Hk, K, V, scale, decay: one chunk, several, shared heads, segments
    (1, 32, 2, 2, 128, 128, 1.0, "token"), (2, 33, 4, 2, 64, 128, -0.3, "token"), (1, 130, 6, 2, 128, 64, 0.3, "head"),
    (2, 300, 3, 3, 128, 128, 0.3, "token"), (1, 700, 2, 1, 32, 32, -0.3, "head"), (1, 1537, 2, 1, 128, 128, 0.3, "token"),
]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,H,Hk,K,V,scale,decay", CASES)
def test_hd_forward_operands(B, T, H, Hk, K, V, scale, decay, io):
    x = hd_inputs(B, T, H, Hk, K, V, io, 300 + T, decay)
    a, dt, n = _abs(x), DT[io], roundings(T, K, V)
    o, _ = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], scale=scale)
    ref, _ = ol.hd_forward(x["q"], x["k"], x["v"], x["g"], x["S0"], None, scale)
    mag, _ = ol.hd_forward(a["q"], a["k"], a["v"], a["g"], a["S0"], None, abs(scale))
    close("o", o, ref, half_step(dt) * ref.abs() + (PAIR[io] + n * U) * mag)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("want_dg", [True, False])
@pytest.mark.parametrize("B,T,H,Hk,K,V,scale,decay", CASES)
def test_hd_gradient_operands(B, T, H, Hk, K, V, scale, decay, want_dg, io):
    if decay == "head" and want_dg:
        want_dg = False  # a constant per head has none
    x = hd_inputs(B, T, H, Hk, K, V, io, 400 + T, decay)
    a, dt, n = _abs(x), DT[io], roundings(T, K, V, H // Hk)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], scale=scale,
                         want_dg=want_dg)
    ref = ol.hd_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"], None, scale)
    mag = ol.hd_backward(a["q"], a["k"], a["v"], a["g"], a["do"], a["S0"], a["dS"], None, abs(scale))
    for name in ("dq", "dk", "dv"):
        close(name, r[name], ref[name], half_step(dt) * ref[name].abs() + (PAIR[io] + n * U) * mag[name])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(97, 3), (700, 1)])
def test_hd_growing_states(T, H, io):
    """Log-decays of both signs, whose sums stay in range: states that grow by up to e^9 over a sequence and shrink again."""
    x = hd_inputs(1, T, H, H, 64, 64, io, 900 + T)
    wave = torch.sin(torch.arange(T, dtype=torch.float32) * (6.3 / T)) * (28.0 / T)
    x["g"] = wave[None, :, None].expand(1, T, H).to(DT[io]).contiguous().cuda()
    a, dt, n = _abs(x), DT[io], roundings(T, 64, 64)
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    (ref, rS), (mag, mS) = (ol.hd_forward(*[y[m] for m in ("q", "k", "v", "g", "S0")]) for y in (x, a))
    close("o", o, ref, half_step(dt) * ref.abs() + (PAIR[io] + n * U) * mag)
    close("S_final", S, rS, n * U * mS)
    r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"])
    ref, mag = (ol.hd_backward(*[y[m] for m in ("q", "k", "v", "g", "do", "S0", "dS")]) for y in (x, a))
    for name in ("dq", "dk", "dv"):
        close(name, r[name], ref[name], half_step(dt) * ref[name].abs() + (PAIR[io] + n * U) * mag[name])
    close("dS0", r["dS0"], ref["dS0"], n * U * mag["dS0"])
