"""GPU tests of rotary positions where values or arguments are unusual."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda
from kda_gated_delta_chunk_amd import _lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BITS = {"bf16": torch.int16, "fp32": torch.int32}


def rnd(shape, seed, dt=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(96, 22), (96, 2), (64, 34), (80, 40), (36, 6), (18, 10), (257, 130), (9, 8)])
def test_copied_channels_keep_their_bits(D, R, layout, io):
    """Channels behind R are copied whatever they hold (infinities, NaN, negative zeros), and reach no others; in place
    too, there they are what they were."""
    q = rnd((5, 3, D), 1, DT[io])
    odd = torch.tensor([float("inf"), float("nan"), -0.0, float("-inf")]).to(q)
    q[..., R:] = odd[torch.arange(D - R, device="cuda") % 4]
    f = kda.rotary_freqs(R)
    clean = q.clone()
    clean[..., R:] = 1.0
    want = kda.rotary(clean, f, layout=layout)
    place = q.clone()
    for y in (kda.rotary(q, f, layout=layout), kda.rotary(place, f, layout=layout, out=place)):
        assert torch.equal(y[..., R:].view(BITS[io]), q[..., R:].view(BITS[io]))
        assert torch.equal(y[..., :R], want[..., :R])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_frequencies_that_are_no_numbers(bad, layout, io):
    """An angle that is no number turns its pair into NaN, at position 0 too, and no other pair."""
    q, f = rnd((4, 3, 40), 1, DT[io]), kda.rotary_freqs(24)
    want = kda.rotary(q, f, layout=layout)
    f[5] = bad
    y = kda.rotary(q, f, layout=layout)
    hit = torch.zeros(40, dtype=torch.bool, device="cuda")
    hit[[5, 17] if layout == "half" else [10, 11]] = True
    assert bool(y[..., hit].isnan().all())
    assert torch.equal(y[..., ~hit], want[..., ~hit])


@pytest.mark.parametrize("T", [1, 3, 9, 10, 11, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40, 2 ** 63 - 1])
def test_period_of_the_positions(T):
    """Without positions a token's is its index modulo T, for any T (the C interface; Python's T is an axis)."""
    n, H, D = 10, 2, 32
    q, f = rnd((n, H, D), 1), kda.rotary_freqs(D)
    y = torch.empty_like(q)
    st = _lib.load().kda_rotary(q.data_ptr(), None, f.data_ptr(), None, y.data_ptr(), None, n, T, H, 0, D, D, 0, 0, 0, 1.0,
                                torch.cuda.current_stream().cuda_stream)
    assert st == 0
    pos = torch.tensor([t % T for t in range(n)], dtype=torch.int32, device="cuda")
    assert torch.equal(y, kda.rotary(q, f, positions=pos))


def test_period_is_ignored_beside_positions():
    q, f = rnd((10, 2, 32), 1), kda.rotary_freqs(32)
    y, pos = torch.empty_like(q), torch.arange(10, dtype=torch.int32, device="cuda") * 7
    for T in (-1, 0, 1, 2 ** 32):
        st = _lib.load().kda_rotary(q.data_ptr(), None, f.data_ptr(), pos.data_ptr(), y.data_ptr(), None, 10, T, 2, 0, 32, 32,
                                    0, 0, 0, 1.0, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(y, kda.rotary(q, f, positions=pos))
