"""The router's workspace without a GPU: its size covers what the kernels write for any batch, one without tokens
among them."""
import pytest

import fp8_fine_grained_fp8q_amd as fq


@pytest.mark.parametrize("E", [1, 16, 64, 65, 256, 257, 1024])
@pytest.mark.parametrize("B", [1, 2, 8, 65535])
def test_room_for_every_workgroup(B, E):
    """A counter (16 bytes), the loss's parts (8 bytes per 64 experts and sequence) and, of every workgroup, E sums,
    E counts and two totals of 4 bytes; a sequence has one workgroup at the least, also without tokens."""
    size = fq.load_library().fp8q_moe_route_workspace
    fixed, each = 16 + 8 * B * -(-E // 64), 4 * B * (2 * E + 2)
    assert size(B, 0, E) == size(B, 1, E) == fixed + each
    at_once = 32 if E <= 256 else 8
    assert size(B, at_once, E) == fixed + each and size(B, at_once + 1, E) == fixed + 2 * each
    if B <= 8:
        assert size(B, 1 << 20, E) == fixed + 256 * each
