"""Int8 stages refuse a routing of other tokens or slots, whose rows lie outside their arrays, before any launch."""

import pytest
import torch

import fp8_block_scaled_moe_amd as fm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K", [(4, 2), (8, 1), (7, 2)])
def test_routing_of_other_rows(T, K):
    E, H, I = 4, 256, 128
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
    r = fm.route_permute(z(8, 2, dtype=torch.int32), E, 16)
    w13, w2 = z(E, 2 * I, H, dtype=torch.int8), z(E, H, I, dtype=torch.int8)
    with pytest.raises(ValueError, match="route"):
        fm.gemm1_swiglu_int8(z(T, H, dtype=torch.int8), z(T), w13, z(E, 2 * I), r, T, K, 16)
    cap = r["sorted_src"].numel()
    with pytest.raises(ValueError, match="route"):
        fm.gemm2_weighted_int8(z(cap, I, dtype=torch.int8), z(cap), w2, z(E, H), r, z(T, K), T, K, 16)


def test_routing_of_the_two_arrays_that_the_stages_read():
    E, H, I, T, K = 4, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    ri = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    x, w13, xs, ws = ri(T, H), ri(E, 2 * I, H), torch.full((T,), 0.01, device="cuda"), torch.full((E, 2 * I), 0.01,
                                                                                                device="cuda")
    r = fm.route_permute(torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32), E, 16)
    part = {k: r[k] for k in ("padded_indptr", "sorted_src")}
    assert torch.equal(fm.gemm1_swiglu_int8(x, xs, w13, ws, part, T, K, 16),
                       fm.gemm1_swiglu_int8(x, xs, w13, ws, r, T, K, 16))
