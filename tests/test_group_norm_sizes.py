"""Workspace sizes of group norm (CPU: the library only computes them)."""
import pytest
import torch

import gated_delta_rule_85_b200 as kda


@pytest.mark.parametrize("C,G", [(65537, 65537), (262147, 262147), (1000003, 1000003), (999999, 333333), (16776959, 16776959)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,L", [(1, 1), (3, 1), (1, 40)])
def test_narrow_groups_take_a_multiple_of_the_tensor(C, G, dtype, N, L):
    """One partial sum (8 bytes) for each group, row tile and one or two channel blocks; gradients add one
    for each channel and row tile.  A row tile is at least 8 positions, or the sample's."""
    tiles = N * -(-L // min(L, 8))
    assert kda.group_norm_workspace_size(N, L, C, G, dtype) <= 2 * 8 * G * tiles
    assert kda.group_norm_workspace_size(N, L, C, G, dtype, backward=True) <= 2 * 8 * G * tiles + 8 * C * tiles


@pytest.mark.parametrize("N,L,C,G", [(1 << 40, 1, 64, 4), ((1 << 24) + 1, 3, 30, 3), (1 << 23, 1, 1024, 256),
                                     (1, 1, 16776961, 1), (1, (1 << 30) + 1, 8, 1)])
def test_sizes_that_are_refused_need_nothing(N, L, C, G):
    """A caller that allocates first gets the refusal, not an allocation that cannot be had."""
    assert kda.group_norm_workspace_size(N, L, C, G) == 0
    assert kda.group_norm_workspace_size(N, L, C, G, backward=True) == 0
    a = [0x10000 * (i + 1) for i in range(12)]   # aligned addresses that nothing dereferences
    lib = kda.load_library()
    assert lib.kda_group_norm_forward(a[0], None, None, None, a[1], a[2], a[3], N, L, C, G, 1e-5, 1, 0, None, 0, None) == -2
    assert "at most" in kda.last_error() or "above" in kda.last_error()
