"""GPU tests of sizes past 32 bits that the library takes as 32-bit numbers: refused (their low bits alone would name other,
valid sizes, and most of a result would stay unwritten). The tensors are never touched."""
import pytest
import torch

import kda_gated_delta_chunk_amd as kda

pytestmark = pytest.mark.gpu

PAST = 1 << 32


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_checkpoints():
    with pytest.raises(ValueError, match="2\\^31"):
        kda.checkpoint8(empty(PAST + 128))
    with pytest.raises(ValueError, match="2\\^31"):
        kda.restore8(kda.Checkpoint8(empty(PAST + 128, dtype=torch.int8), empty((PAST + 128) // 128, dtype=torch.float32),
                                     torch.bfloat16))


def test_norms():
    x = empty(1, PAST + 64)
    for call in (lambda: kda.layer_norm_fwd(x), lambda: kda.layer_norm_bwd(x, x)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_rotations():
    q, freqs = empty(1, 1, PAST + 32), kda.rotary_freqs(32)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.rotary(q, freqs)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.rotary_axes(q, freqs, kda.rotary_sections([8, 8]), torch.zeros((2, 1), dtype=torch.int32, device="cuda"))


def test_recurrences():
    q, v, g = empty(1, 1, 1, PAST + 32), empty(1, 1, 1, 32), empty(1, 1, 1)
    S = torch.zeros((1, 1, 32, 32), device="cuda")
    for call in (lambda: kda.gd_chunk_fwd(q, q, v, g, g), lambda: kda.gd_chunk_bwd(q, q, v, g, g, v),
                 lambda: kda.gd_decode_step(q[0], q[0], v[0], g[0], g[0], S), lambda: kda.hd_chunk_fwd(q, q, v, g),
                 lambda: kda.hd_chunk_bwd(q, q, v, g, v), lambda: kda.hd_decode_step(q[0], q[0], v[0], g[0], S)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_many_rows_are_no_such_size():
    """2^31 rows and more are counted in 64 bits."""
    x = empty((1 << 31) + 5, 1).fill_(1.5)
    x[-1] = -3.0
    y = kda.restore8(kda.checkpoint8(x))
    assert float(y[0]) == 1.5 and float(y[-1]) == -3.0 and float(y[1 << 31]) == 1.5
