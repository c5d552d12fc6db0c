"""CPU tests of what the gated delta rule's gradients ask for as workspace: states only where one segment of a sequence hands
over to the next (16 chunks of 32 tokens at 96 heads of 128 channels)."""
import kda_gated_delta_chunk_amd as kda

H, K, V, CHUNK, SEGMENT = 96, 128, 128, 32, 512
STATE = H * K * V * 4
# bf16 I/O, of one chunk: three matrices of 4096 bytes and a third part of 2048 each, 8 rows of 32 weights, and the two tiles of
# the walks in three bf16 parts
PER_CHUNK = H * (3 * (4096 + 2048) + 8 * CHUNK * 4 + 2 * V * CHUNK * 6)
PER_TOKEN = H * K * 4  # dk's first part
ROUND = 1 << 12  # every part begins on a multiple of 256 bytes


def asks(B, T, num_seqs=None, packed=False):
    return kda.gd_bwd_workspace_bytes(B, T, H, K, V, num_seqs or B, packed=packed)


def test_rows_of_one_segment_keep_no_states():
    for B, T in ((1, 1), (7, 100), (64, SEGMENT)):
        chunks = B * -(-T // CHUNK)
        assert 0 < asks(B, T) <= chunks * PER_CHUNK + B * T * PER_TOKEN + ROUND


def test_a_border_keeps_two():
    for B, T in ((1, SEGMENT + 1), (3, 4 * SEGMENT), (1, 4096)):
        rest = B * (-(-T // CHUNK) * PER_CHUNK + T * PER_TOKEN)
        states = 2 * STATE * B * ((T - 1) // SEGMENT)
        assert 0 < asks(B, T) <= rest + states + ROUND


def test_packed_sequences_keep_what_their_tokens_can_need():
    """N sequences have at most T / 512 borders, however many they are, and T / 32 + N chunks."""
    for T, N in ((512 * 32, 512), (17011, 16), (500, 400)):
        rest = (T // CHUNK + N) * PER_CHUNK + T * PER_TOKEN
        states = 2 * STATE * (T // SEGMENT)
        assert asks(1, T, N, True) <= rest + states + 64 * N + ROUND
