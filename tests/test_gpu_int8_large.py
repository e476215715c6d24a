"""Int8 stages and the combine where a launch has more workgroups than one grid dimension takes (2^32 threads).  The
GEMMs give the same bits as with tall tiles, which need few workgroups."""

import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def test_streaming_gemm1_of_many_workgroups():
    """262160 rows of 1024 N tiles, 16 rows a tile."""
    T, H, I = (1 << 18) + 16, 128, 16384
    say("int8 gemm1 workgroups", T, H, I)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-127, 128, (T, H), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (1, 2 * I, H), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(T, generator=g, device="cuda") * 0.01
    ws = torch.rand(1, 2 * I, generator=g, device="cuda") * 0.01
    r = fm.route_permute(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1, 16)
    tall = fm.gemm1_swiglu_int8(x, xs, w, ws, r, T, 1, 16, tile_m=288)
    short = fm.gemm1_swiglu_int8(x, xs, w, ws, r, T, 1, 16, tile_m=16)
    torch.cuda.synchronize()
    for a in range(0, T, 1 << 16):
        assert torch.equal(short[a:a + (1 << 16)], tall[a:a + (1 << 16)])


def test_streaming_gemm2_of_many_workgroups():
    """524304 rows of 512 N tiles, 16 rows a tile."""
    T, H, I = (1 << 19) + 16, 16384, 128
    say("int8 gemm2 workgroups", T, H, I)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(-127, 128, (1, H, I), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(1, H, generator=g, device="cuda") * 0.01
    r = fm.route_permute(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1, 16)
    cap = r["sorted_src"].numel()
    q = torch.randint(-127, 128, (cap, I), generator=g, device="cuda", dtype=torch.int8)
    qs = torch.rand(cap, generator=g, device="cuda") * 0.01
    tw = torch.rand(T, 1, generator=g, device="cuda")
    tall = fm.gemm2_weighted_int8(q, qs, w, ws, r, tw, T, 1, 16, tile_m=288)
    short = fm.gemm2_weighted_int8(q, qs, w, ws, r, tw, T, 1, 16, tile_m=16)
    torch.cuda.synchronize()
    for a in range(0, T, 1 << 16):
        assert torch.equal(short[a:a + (1 << 16)], tall[a:a + (1 << 16)])


def test_combine_of_many_tokens():
    """2^24 + 5 tokens, of 256 threads each."""
    T, H = (1 << 24) + 5, 128
    say("combine tokens", T, H)
    Y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    for a in range(0, T, 1 << 20):
        Y[a:a + (1 << 20)] = (torch.arange(a, min(a + (1 << 20), T), device="cuda") % 251)[:, None] + 1
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[::3] = -1
    out = fm.combine(Y, ids, 1)
    torch.cuda.synchronize()
    Y[::3] = 0
    for a in range(0, T, 1 << 20):
        assert torch.equal(out[a:a + (1 << 20)], Y[a:a + (1 << 20)])
