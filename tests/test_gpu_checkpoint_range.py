"""GPU tests of the checkpoints in 8 bits at the ends of their types' ranges.

A value is a code times a scale, both rounded to fp32: besides half a scale it is off by 127 steps' roundings of 2^-24 each,
and by those of the code's product and quotient, 4 * 127 * 2^-24 < 2^-14 of a scale together; bf16 adds half its own step."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from oracle import layers as ol
from tests.test_gpu_layers import DT, close, half_step, rnd

pytestmark = pytest.mark.gpu


def ends(io, shape, seed):
    """Rows of ordinary and of large values, some blocks of which hold the type's largest, of either sign, or one next to it."""
    dt = DT[io]
    most = torch.finfo(dt).max
    x = rnd(shape, seed, dt).clamp(-8, 8)
    x[1::2] *= 2.0 ** 122
    x[1, 3], x[2, -1], x[3] = most, -most, -most  # a row of the usual mask value
    if io == "fp32":
        for i in range(1, 40):  # the values next to it
            x[4 + i % 3, (7 * i) % shape[1]] = torch.tensor(most).view(torch.int32).sub(i).view(torch.float32)
    return x


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [7, 100, 128, 513, 1024])
def test_the_largest_values(C, io):
    x = ends(io, (9, C), 3)
    c = kda.checkpoint8(x)
    y = kda.restore8(c)
    assert bool(x.isfinite().all()) and bool(c.scales.isfinite().all())
    step = c.scales.double().cpu().repeat_interleave(128, dim=1)[:, :C]
    close("restored", y, ol.f64(x), (0.5 + 2.0 ** -14) * step + (half_step(DT[io]) * y.double().abs().cpu() if io == "bf16" else 0.0))
    # the values that a gradient reads out of the codes are the same
    dy, w = rnd((9, C), 5, DT[io]), rnd((C,), 6)
    got, want = kda.layer_norm_bwd(dy, c, weight=w), kda.layer_norm_bwd(dy, y, weight=w)
    for n in want:
        assert torch.equal(got[n].nan_to_num(nan=7.0), want[n].nan_to_num(nan=7.0)), n


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_scales_are_the_quotient_wherever_it_holds(io):
    """max / 127 in fp32, from 2^-119 to where 127 of it would pass the largest value."""
    top = torch.exp2(torch.linspace(-119, 127.9, 4001)).to(DT[io])
    x = torch.zeros((4001, 40), dtype=DT[io])
    x[:, 11] = -top
    scales = kda.checkpoint8(x.cuda()).scales.cpu()[:, 0]
    assert torch.equal(scales, top.float() / 127.0)
