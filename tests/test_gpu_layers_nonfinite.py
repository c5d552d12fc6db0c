"""GPU tests of linear attention with one decay per head on inputs with NaN and infinities: what does not depend on such
a value by the definition (oracle.layers, fp64) is what it is without it. Garbage behind a prompt that shares its row is
the everyday case."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import layers as ol
from tests.test_gpu_layers import DT, _abs, close, half_step, hd_inputs
from tests.test_gpu_layers_operands import PAIR, roundings, U

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def finite_agree(name, got, ref, mag, io, n):
    """Where the definition's result is finite: close to it. (Where it is not, the kernels may give any such value.)"""
    live = ref.isfinite() & mag.isfinite()
    got = got.cpu()
    close(name, got[live], ref[live], (half_step(DT[io]) * ref.abs() + (PAIR[io] + n * U) * mag)[live])
    assert not bool(got[~ref.isfinite()].isfinite().any()), name


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [32, 61, 100])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("q", -INF), ("g", NAN)])
@pytest.mark.parametrize("at", [0, 7, 15, 16, 31])
def test_hd_forward_is_causal(at, name, value, T, io):
    """One such entry at a token of the last chunk: the outputs before it, and of other columns, do not see it."""
    x = hd_inputs(1, T, 2, 2, 64, 64, io, 500 + T)
    t = min((T - 1) // 32 * 32 + at, T - 1)
    if name == "g":
        x["g"][0, t, 1] = value
    else:
        x[name][0, t, 1, 37] = value
    o, S = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    ref, rS = ol.hd_forward(x["q"], x["k"], x["v"], x["g"], x["S0"])
    a = _abs(x)
    mag, mS = ol.hd_forward(a["q"], a["k"], a["v"], a["g"], a["S0"])
    n = roundings(T, 64, 64)
    finite_agree("o", o, ref, mag, io, n)
    finite_agree("o", o[:, :t], ref[:, :t], mag[:, :t], io, n)
    assert bool(ref[:, :t].isfinite().all())
    live = rS.isfinite() & mS.isfinite()
    close("S_final", S.cpu()[live], rS[live], (n * U * mS)[live])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(32, 128), (128, 32), (128, 128)])
def test_hd_garbage_behind_a_prompt(K, V, io):
    """Prompts of several lengths in rows of one batch, garbage behind them: their outputs are those of clean rows."""
    T, lengths = 200, [5, 32, 47, 170]
    x = hd_inputs(4, T, 3, 1, K, V, io, 600)
    ref, _ = ol.hd_forward(x["q"], x["k"], x["v"], x["g"], x["S0"])
    a = _abs(x)
    mag, _ = ol.hd_forward(a["q"], a["k"], a["v"], a["g"], a["S0"])
    for b, n in enumerate(lengths):
        for name in ("q", "k", "v", "g"):
            x[name][b, n:] = NAN if b % 2 else INF
    o, _ = kda.hd_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    for b, n in enumerate(lengths):
        close("o", o[b, :n], ref[b, :n], (half_step(DT[io]) * ref.abs() + (PAIR[io] + roundings(T, K, V) * U) * mag)[b, :n])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [32, 61, 100])
@pytest.mark.parametrize("name,value", [("v", NAN), ("k", INF), ("q", NAN), ("do", NAN), ("do", -INF)])
@pytest.mark.parametrize("at", [0, 7, 16, 31])
def test_hd_gradients_reach_what_depends(at, name, value, T, io):
    """dq sees k and v up to its token, dk and dv see q and do from theirs on; dg is summed over a head's tokens and may
    be spoiled throughout."""
    x = hd_inputs(1, T, 2, 2, 64, 64, io, 700 + T)
    t = min((T - 1) // 32 * 32 + at, T - 1)
    x[name][0, t, 1, 37] = value
    a = _abs(x)
    ref = ol.hd_backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"])
    mag = ol.hd_backward(a["q"], a["k"], a["v"], a["g"], a["do"], a["S0"], a["dS"])
    for want_dg in (True, False):
        r = kda.hd_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_final=x["dS"], want_dg=want_dg)
        for res in ("dq", "dk", "dv"):
            finite_agree(res, r[res], ref[res], mag[res], io, roundings(T, 64, 64))
        assert bool(ref["dg"][:, :, 0].isfinite().all())
        if want_dg:
            assert bool(r["dg"][:, :, 0].isfinite().all())
