"""The int8 layer's workspace: one made for the largest batch serves every smaller one.  No GPU is touched."""

import pytest

import fp8_block_scaled_moe_amd as fm


@pytest.mark.parametrize("H,I,E,K", [(1024, 128, 16, 4), (7168, 2048, 256, 8), (2048, 768, 128, 8), (128, 128, 1, 1)])
def test_workspace_grows_with_the_tokens(H, I, E, K):
    border = (1 << 22) // (H * K)      # T * K * H = 2^22 values of Y
    sizes = [fm.fused_int8_workspace_size(T, H, I, E, K)
             for T in (0, 1, border // 2, border - 1, border, border + 1, border + 2, 2 * border, 2 * border + 1, 5 * border)]
    assert sizes == sorted(sizes)
