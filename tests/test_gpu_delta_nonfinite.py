"""GPU tests of the gated delta rule with values that are not finite, over every pair of types: the kernels beside fp32 gates
take their operands in three bf16 parts, those beside bf16 gates in two. Tolerances as in test_gpu_delta, where the definition
is clean: the tokens that do not depend on the value."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import delta as od
from tests.test_gpu_delta import ARGS, INF, NAN, finite_agree, inputs

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]


@pytest.mark.parametrize("io,gates", TYPES)
@pytest.mark.parametrize("K,V,T", [(64, 64, 61), (128, 128, 100)])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("k", INF), ("q", NAN), ("do", NAN), ("do", -INF)])
@pytest.mark.parametrize("at", [0, 7, 16, 21])
def test_gradients_before_and_behind(at, name, value, K, V, T, io, gates):
    """What include/kda.h says of each: a v reaches dq and dk from its token on and no dv, a q dk and dv up to its token and no
    other dq, a d_o the same and its own dq, a k dq from its token on and dv up to it. (A dg or dbeta may be spoiled.) The
    tokens beside the value share a register with it: even and odd ones are asked."""
    x = inputs(1, T, 4, 2, K, V, io, 800 + T, gates)
    t = min((T - 1) // 32 * 32 + at, T - 2)
    clean, far = od.gd_backward(*(x[n] for n in ARGS), x["do"], x["S0"], x["dS"], spread=True)
    if name in ("q", "k"):
        x[name][0, t, 1, 37] = value  # of heads 2 and 3
    else:
        x[name][0, t, 2, 37] = value
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    reaches = {"v": {"dq": slice(0, t), "dk": slice(0, t), "dv": slice(0, T)},
               "q": {"dk": slice(t + 1, T), "dv": slice(t + 1, T)}, "do": {"dk": slice(t + 1, T), "dv": slice(t + 1, T)},
               "k": {"dq": slice(0, t), "dv": slice(t + 1, T)}}[name]
    for n, rest in reaches.items():
        finite_agree(n, r[n][:, rest], clean[n][:, rest], far[n][:, rest], x)
    if name in ("q", "do"):  # dq_t = S do_t: no other row, of a q not its own either
        for rest in (slice(0, t), slice(t + (name == "do"), T)):
            finite_agree("dq", r["dq"][:, rest], clean["dq"][:, rest], far["dq"][:, rest], x)
    for n in ("dq", "dk"):
        finite_agree(n + " of other heads", r[n][:, :, :1], clean[n][:, :, :1], far[n][:, :, :1], x)
    for n in ("dv", "dg", "dbeta"):
        finite_agree(n + " of other heads", r[n][:, :, :2], clean[n][:, :, :2], far[n][:, :, :2], x)


@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("q", -INF), ("g", NAN), ("beta", INF)])
@pytest.mark.parametrize("at", [0, 7, 16, 31])
@pytest.mark.parametrize("T", [61, 100])
def test_forward_is_causal_beside_fp32_gates(T, at, name, value):
    x = inputs(1, T, 2, 2, 64, 64, "bf16", 900 + T, "fp32")
    t = min((T - 1) // 32 * 32 + at, T - 1)
    clean, _, far, _ = od.gd_forward(*(x[n] for n in ARGS), x["S0"], spread=True)
    if name in ("g", "beta"):
        x[name][0, t, 1] = value
    else:
        x[name][0, t, 1, 37] = value
    o, _ = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    bad = ~od.gd_forward(*(x[n] for n in ARGS), x["S0"])[0].isfinite()
    assert bool(bad.any()) and not bool(bad[:, :t].any()) and not bool(bad[:, :, 0].any())
    assert not bool(o.cpu()[bad].isfinite().any())
    finite_agree("o", o[~bad], clean[~bad], far[~bad], x)


@pytest.mark.parametrize("K,V", [(64, 128), (128, 128)])
def test_garbage_behind_a_prompt_beside_fp32_gates(K, V):
    T, lengths = 200, [5, 32, 47, 170]
    x = inputs(4, T, 3, 1, K, V, "bf16", 950, "fp32")
    ref, _, far, _ = od.gd_forward(*(x[n] for n in ARGS), x["S0"], spread=True)
    for b, n in enumerate(lengths):
        for name in ARGS:
            x[name][b, n:] = NAN if b % 2 else INF
    o, _ = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"])
    for b, n in enumerate(lengths):
        finite_agree("o", o[b, :n], ref[b, :n], far[b, :n], x)
