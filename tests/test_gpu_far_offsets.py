"""Norm, router and int8 layer where offsets pass 32 bits: the last rows of a large call give the bits of a call on
those rows alone (of enough rows that both take the same kernels)."""

import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [fm.NORM_FP8, fm.NORM_MXFP8, fm.NORM_INT8])
def test_norm(fmt):
    """2^32 values and more."""
    T, H, n = (1 << 18) + 77, 16384, 600
    say("norm far", fmt)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    r = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(H, generator=g, device="cuda")
    big = fm.add_rmsnorm_quant(x, w, 1e-6, fmt, residual=r, want_norm=True)
    part = fm.add_rmsnorm_quant(x[-n:], w, 1e-6, fmt, residual=r[-n:], want_norm=True)
    torch.cuda.synchronize()
    for a, b in zip(big, part):
        assert torch.equal(a[-n:], b)


@pytest.mark.parametrize("biased", [False, True])
def test_router(biased):
    """More than 2^32 bytes and 2^31 values of logits."""
    T, E, K, n = (1 << 21) + 33, 1024, 8, 17000
    say("router far", biased)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(T, E, device="cuda").normal_(generator=g)
    kw = dict(bias=0.1 * torch.randn(E, generator=g, device="cuda"), n_group=8, topk_group=4, group_top=2) if biased else {}
    ids, weights = fm.moe_router_topk(x, K, **kw)
    ids2, weights2 = fm.moe_router_topk(x[-n:], K, **kw)
    torch.cuda.synchronize()
    assert torch.equal(ids[-n:], ids2) and torch.equal(weights[-n:], weights2)


@pytest.mark.parametrize("packed", [False, True])
def test_int8_layer(packed):
    """Tokens of 4 GiB and more: GEMM1 leaves the tile kernel, whose token offsets have 32 bits."""
    T, H, I, E, n = (1 << 18) + 50, 16384, 128, 2, 900
    say("int8 far", packed)
    g = torch.Generator(device="cuda").manual_seed(3)
    ri = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    x, w13, w2 = ri(T, H), ri(E, 2 * I, H), ri(E, H, I)
    if packed:
        w13, w2 = fm.pack_weights(w13), fm.pack_weights(w2)
    xs = torch.rand(T, generator=g, device="cuda") * 0.01
    w13s, w2s = (torch.rand(E, m, generator=g, device="cuda") * 1e-3 for m in (2 * I, H))
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    tw = torch.rand(T, 1, generator=g, device="cuda")
    out = fm.moe_fused_int8(x, xs, w13, w13s, w2, w2s, ids, tw, weight_layout=int(packed))
    part = fm.moe_fused_int8(x[-n:], xs[-n:], w13, w13s, w2, w2s, ids[-n:], tw[-n:], weight_layout=int(packed))
    torch.cuda.synchronize()
    assert torch.equal(out[-n:], part)
    assert out[:n].abs().sum() > 0
