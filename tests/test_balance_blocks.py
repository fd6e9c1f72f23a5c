"""Tokens of a block of the losses' kernel, by the workspace's size (two slots of
E sums and E counts, and a sum, for each block): whole rounds of its 16 warps, of
which each takes as many tokens at once as their lanes (E / 4, rounded up to a
power of two from 4 to 32) fit in it."""
import pytest

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build


@pytest.mark.parametrize("E", [1, 8, 16, 17, 20, 21, 24, 32, 33, 40, 41, 48, 63, 64, 65, 96, 128, 129, 256, 300, 1024])
def test_whole_rounds(E):
    build()
    lanes = 4
    while lanes < 32 and 4 * lanes < E:
        lanes *= 2
    at_once = 16 * (32 // lanes)
    for rounds in (1, 2, 3, 7):
        T = 304 * rounds * at_once  # two blocks an SM, all of them full
        size = B.dwdp_balance_workspace_bytes(T, E, 1)
        assert size == 304 * (2 * E * 8 + 8)
        # one token more: a round more for each block
        T += 1
        blocks = -(-T // ((rounds + 1) * at_once))
        assert B.dwdp_balance_workspace_bytes(T, E, 1) == blocks * (2 * E * 8 + 8)
