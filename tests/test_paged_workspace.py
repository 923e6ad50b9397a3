"""CPU checks of how large a workspace msa_paged_attend asks for."""
import pytest


@pytest.fixture(scope="module")
def size():
    from routed_kv_memory_amd import msa
    msa.lib()
    return msa.msa_paged_attend_workspace_size


@pytest.mark.parametrize("layers,B,groups,tokens,hq", [
    (18, 16, 1, 16, 32), (18, 64, 8, 64, 32), (18, 256, 256, 256, 32), (18, 2048, 256, 2048, 32), (36, 2048, 2, 2048, 64),
    (1, 64, 64, 64, 8), (64, 700, 100, 900, 16)])
def test_decode_steps(size, layers, B, groups, tokens, hq):
    """A part of a column is 128 dims, its maximum and sum.  A step writes at most one of every column's own rows
    and one of its group's, and those of the rows that are cut (128 columns for each of the workgroups aimed at, in
    streams 64).  Room: streams of up to 16 columns take 16 in 8 heads, for every sequence and for the
    rows that two or more share; shared columns in tiles take up to twice as many, as own ones would.  A layer's
    plan is 256 threads' of under 256 bytes."""
    part, G = 4 * 128 + 8, hq // 8
    streams, tiles, cut = 8 * 16 * (B + B // 2), 8 * 2 * 2 * G * tokens, (max(512 // layers, 56) + 1) * (128 + 64)
    assert size(layers, B, groups, tokens, hq) <= layers * (part * (streams + tiles + cut) + 64 * tokens + (1 << 16)) + (1 << 12)


def test_one_sequence_shares_with_none(size):
    """A prompt's parts are those of the rows that are cut, however many tokens it has."""
    assert size(1, 1, 1, 8000, 32) < 60e6
    assert size(1, 1, 1, 1 << 20, 32) - size(1, 1, 1, 1 << 19, 32) == (1 << 19) * 64        # where the parts are


def test_long_sequences_share_nothing(size):
    """Sequences of more than 512 columns read their rows themselves: 8 prompts need about what 2 groups of them do."""
    assert size(4, 8, 8, 8704, 32) < 0.25e9
    assert size(1, 8, 2, 8000, 32) < 0.1e9
