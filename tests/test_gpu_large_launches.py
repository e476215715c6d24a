"""GEMMs of so many rows that their short tiles would take more than 2^32 threads: the same bits as with tall ones."""

import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def test_fp8_gemm1_of_many_workgroups():
    """1048592 rows of 128 N tiles, 16 rows a tile."""
    T, H, I = (1 << 20) + 16, 128, 16384
    say("fp8 gemm1 workgroups", T, H, I)
    g = torch.Generator(device="cuda").manual_seed(1)
    code = lambda *s: torch.randint(0, 0x7F, s, generator=g, device="cuda", dtype=torch.uint8)
    x, w = code(T, H), code(1, 2 * I, H)
    xs = torch.rand(T, 1, generator=g, device="cuda") * 1e-3
    ws = torch.rand(1, 2 * I // 128, 1, generator=g, device="cuda") * 1e-3
    r = fm.route_permute(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1, 16)
    q, s = fm.gemm1_swiglu_quant(x, xs, w, ws, r, T, 1, 16, tile_m=128)
    q2, s2 = fm.gemm1_swiglu_quant(x, xs, w, ws, r, T, 1, 16, tile_m=16)
    torch.cuda.synchronize()
    for a in range(0, T, 1 << 17):
        b = a + (1 << 17)
        assert torch.equal(q[a:b], q2[a:b]) and torch.equal(s[a:b], s2[a:b])
