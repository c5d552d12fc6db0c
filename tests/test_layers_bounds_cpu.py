"""CPU tests of the size limits of the operators around the recurrence: sizes whose grids would not fit are refused before
anything touches a device, and the largest that fit are not."""
import math

import pytest

from kda_gated_delta_chunk_amd import _lib

INVALID = 1
A, M = 1 << 20, 1 << 40  # addresses that are never read, ranges apart


def norm_fwd(rows, G, C):
    return _lib.load().kda_layer_norm_fwd(A, A + M, A + 2 * M, None, A + 3 * M, rows, G, C, 1e-5, 1, 1, None)


def norm_bwd(rows, G, C):
    return _lib.load().kda_layer_norm_bwd(A, A + M, A + 2 * M, A + 3 * M, None, A + 4 * M, A + 5 * M, A + 6 * M, None, rows,
                                          G, C, 1e-5, 1, 1, A + 7 * M, 1 << 39, None)


# An odd number of groups needs as many workgroups as groups, of 256 threads at these widths (32 rows a workgroup of up to
# 64 channels): 2^24 of them are 2^32 threads.
@pytest.mark.parametrize("G,C", [(2 ** 25 + 1, 1), (2 ** 24 + 1, 1), (2 ** 24 + 1, 7), (2 ** 27 - 1, 1), (2 ** 25 + 2, 3)])
def test_norm_grids_past_32_bits_are_refused(G, C):
    assert G // math.gcd(G, 32) * 256 >= 2 ** 32
    assert norm_fwd(G, G, C) == INVALID
    assert norm_bwd(G, G, C) == INVALID
    assert _lib.load().kda_layer_norm_bwd_workspace_bytes(G, G, C) == 0


@pytest.mark.parametrize("G,C", [(2 ** 24 - 1, 8), (2 ** 27, 1), (2 ** 26, 2), (2 ** 24, 8), (2 ** 23 + 1, 9), (1, 16384),
                                 (2 ** 17 - 1, 1024), (8191, 16384)])
def test_norm_grids_of_32_bits_are_not(G, C):
    n = _lib.load().kda_layer_norm_bwd_workspace_bytes(G, G, C)
    assert n >= G * C * 8
