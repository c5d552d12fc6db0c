"""GPU tests of the gated delta rule's gradients over segments of every length, against the fp64 definition. A segment is 16
chunks of 32 tokens where H * K is 8192 or more (8 for K below 128), half of it for half of that, 2 at the least. Heads do not
see each other: the definition is asked for those of some q/k heads. Tolerances as in test_gpu_delta."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import delta as od
from tests.test_gpu_delta import ARGS, check_bwd, check_fwd, inputs
from tests.test_gpu_layers import DT, U

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]
GRADS = ("dq", "dk", "dv", "dg", "dbeta")


def segment_tokens(H, K):
    seg = 16 if K == 128 else 8
    while seg > 2 and seg * 512 > H * K:
        seg //= 2
    return 32 * seg


def some_heads(x, r, Hk, group):
    """The inputs and results of three q/k heads and the v heads that share them."""
    few = sorted({0, Hk // 2, Hk - 1})
    v = [h * group + i for h in few for i in range(group)]
    cut = {n: t[:, :, few if n in ("q", "k") else v] if n not in ("S0", "dS") else t[:, v] for n, t in x.items()}
    res = {n: t[:, :, few if n in ("dq", "dk") else v] if n not in ("dS0", "S") else t[:, v] for n, t in r.items()}
    return {n: t.contiguous() for n, t in cut.items()}, res


@pytest.mark.parametrize("io,gates", TYPES)
@pytest.mark.parametrize("chunks,more", [(1, -1), (1, 0), (1, 1), (2, 37)])
@pytest.mark.parametrize("H,Hk,K,V", [(64, 64, 128, 128), (64, 32, 128, 64), (64, 64, 128, 32), (32, 16, 128, 128),
                                      (128, 128, 64, 128), (256, 128, 32, 64), (16, 16, 128, 64)])
def test_borders(H, Hk, K, V, chunks, more, io, gates):
    """One token less than a segment, a whole one, one more, and two with an odd rest."""
    T = chunks * segment_tokens(H, K) + more
    x = inputs(1, T, H, Hk, K, V, io, 40 + T, gates)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], scale=0.3)
    check_bwd(*some_heads(x, r, Hk, H // Hk), scale=0.3)


@pytest.mark.parametrize("io,gates", TYPES)
@pytest.mark.parametrize("T", [65, 97, 128, 300, 500])
def test_walks_of_few_to_many_chunks(T, io, gates):
    """Three chunks, four, ... of one segment: the rows of two chunks at a time turn about in LDS."""
    x = inputs(1, T, 64, 64, 128, 128, io, 60 + T, gates)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    check_bwd(*some_heads(x, r, 64, 1))


@pytest.mark.parametrize("io,gates", TYPES)
@pytest.mark.parametrize("H,Hk,K", [(160, 80, 128), (144, 144, 64), (132, 33, 32)])
def test_both_column_tiles_in_a_workgroup(H, Hk, K, io, gates):
    """More column tiles of 64 than compute units, many chunks: the forward call and the gradients."""
    x = inputs(1, 333, H, Hk, K, 128, io, 65, gates)
    o, S = kda.gd_chunk_fwd(*(x[n] for n in ARGS), S0=x["S0"], scale=0.3)
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], scale=0.3)
    few, res = some_heads(x, {**r, "o": o, "S": S}, Hk, H // Hk)
    check_fwd(few, res["o"], res["S"], scale=0.3)
    check_bwd(few, res, scale=0.3)


@pytest.mark.parametrize("io,gates", TYPES)
def test_packed(io, gates):
    """Sequences of none, one, two and three segments, borders inside chunks."""
    cu, T, H = [3, 515, 515, 516, 1029, 2090, 2100], 2111, 64
    N = len(cu) - 1
    x = inputs(1, T, H, H, 128, 32, io, 71, gates, N=N)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=c)
    check_bwd(*some_heads(x, r, H, 1), cu=c.cpu())


@pytest.mark.parametrize("H,K,V,T", [(4, 128, 128, 700), (64, 128, 128, 1100), (32, 64, 64, 600), (128, 32, 128, 300)])
def test_operands_beside_fp32_gates_keep_their_bits(H, K, V, T):
    """Beside fp32 gates the gradients of bf16 inputs are those of fp32 operands. 2-norms: roundings that are independent of
    each other, 16 of 2^-24 for a row and for a product of rows (dS0, dbeta); dg is a difference of sums over a sequence, four
    times as much. Two bf16 parts in place of three, 2^-18 or 64 such roundings of an operand at most, do not stay within
    this."""
    x = inputs(1, T, H, H, K, V, "bf16", 81, "fp32")
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"])
    x, r = some_heads(x, r, H, 1)
    ref = od.gd_backward(*(x[n] for n in ARGS), x["do"], x["S0"], x["dS"])
    off = {n: float((r[n].cpu().double() - ref[n]).norm() / ref[n].norm()) for n in ("dS0", "dbeta", "dg")}
    assert off["dS0"] < 16 * U and off["dbeta"] < 16 * U and off["dg"] < 64 * U, off


def test_a_sequence_s_segments_are_its_own():
    """Several segments in a packed batch: the same bits as alone."""
    H, K, V, cu = 64, 128, 64, [0, 700, 1300, 2400]
    x = inputs(1, cu[-1], H, H // 2, K, V, "bf16", 91, "fp32", N=3)
    dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = kda.gd_chunk_bwd(*(x[n] for n in ARGS), x["do"], S0=x["S0"], dS_final=x["dS"], cu_seqlens=dev)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        one = [x[m][:, a:b].contiguous() for m in ARGS + ("do",)]
        alone = kda.gd_chunk_bwd(*one, S0=x["S0"][n:n + 1].contiguous(), dS_final=x["dS"][n:n + 1].contiguous())
        for m in GRADS:
            assert torch.equal(r[m][:, a:b], alone[m]), m
        assert torch.equal(r["dS0"][n:n + 1], alone["dS0"])
        assert all(r[m].dtype is DT["fp32"] for m in ("dg", "dbeta"))
