"""quant_fp8_blocks on the GPU against the float64 oracle.

Tolerances.  Plain: the scale is one fp32 division of an exact maximum, within 2^-24 relative (and half a subnormal
step); the quotient v * (448 / amax) carries two roundings, so a code must be the rounding of a value within 3 * 2^-24
of v / scale.  Gated: silu(g) * u is within (2 |g| + 8) 2^-24 relative (device_common.h), |g| <= 87; blocks whose
largest value is below 2^-60 are evaluated in fp64 and rounded once.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle.products import quant_blocks, silu_mul
from tests.gpu_helpers import e4m3_rounding_interval, say

pytestmark = pytest.mark.gpu


def run(x, gated=False, **kw):
    q, s = fm.quant_fp8_blocks(x.cuda(), gated=gated, **kw)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def check(x, gated, q, s):
    v = silu_mul(x.double().numpy()) if gated else x.double().numpy()
    rel = np.full(v.shape, 2.0 ** -23)
    if gated:
        rel += (2 * np.minimum(np.abs(x.double().numpy()[:, :v.shape[1]]), 90) + 8) * 2.0 ** -24
    M, N = v.shape
    col = np.arange(N) // 128
    _, want = quant_blocks(v)
    top = np.stack([np.max(np.where(col == k, rel, 0), axis=1) for k in range(want.shape[1])], 1)
    ok = np.abs(s - want) <= want * (top + 2.0 ** -23) + 2.0 ** -149
    assert np.all(ok), (s[~ok][:4], want[~ok][:4])
    scale = s.astype(np.float64)[:, col]
    exact = v / scale
    lo, hi = e4m3_rounding_interval(q)
    slack = np.abs(exact) * (rel + 3 * 2.0 ** -24) + 2.0 ** -148 / scale
    assert np.all((exact >= lo - slack) & (exact <= hi + slack))


@pytest.mark.parametrize("M,N", [(1, 16), (1, 7168), (3, 112), (5, 128), (7, 144), (33, 400), (64, 2048), (257, 272),
                                 (1000, 1040)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gated", [False, True])
def test_quant(M, N, dtype, gated):
    g = torch.Generator().manual_seed(M + N)
    x = (torch.randn(M, 2 * N if gated else N, generator=g) * 2).to(dtype)
    say("quant", M, N, dtype, gated)
    check(x, gated, *run(x, gated))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wide_range_and_zero_blocks(dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 640, generator=g)
    x *= torch.exp2(torch.randint(-120, 120, (40, 5), generator=g).float()).repeat_interleave(128, 1)
    x[3, 128:256] = 0
    x[4] = 0
    x[5, :128] = 2.0 ** -126
    x = x.to(dtype)
    q, s = run(x)
    check(x, False, q, s)
    assert s[3, 1] == 1 and not q[3, 128:256].any() and np.all(s[4] == 1) and not q[4].any()


def test_subnormal_blocks():
    x = torch.zeros(3, 256)
    x[0, 5] = 2.0 ** -149            # its scale underflows: 1, codes 0
    x[1, 7], x[1, 8] = 2.0 ** -135, 2.0 ** -136
    x[2, 200] = 2.0 ** -127
    q, s = run(x)
    assert s[0, 0] == 1 and not q[0].any()
    check(x[1:], False, q[1:], s[1:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gated_far_negative_gates(dtype):
    """Blocks of gates far below -87, where exp(-gate) leaves fp32: values below 2^-60 come from fp64."""
    x = torch.ones(4, 512)
    x[0, :128], x[1, :128], x[2, :128] = -80.0, -90.0, -102.0
    x[2, 256:384] = 1e30
    x[3, :256] = -1000.0
    x = x.to(dtype)
    q, s = run(x, True)
    check(x, True, q, s)
    assert s[3, 0] == 1 and not (q[3] & 0x7F).any()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_blocks_without_numbers(gated, bad):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 768 if gated else 384, generator=g).bfloat16()
    clean = x.clone()
    x[2, 130] = bad
    x[4, 383] = bad
    q, s = run(x, gated)
    q0, s0 = run(clean, gated)
    hit = np.zeros(s.shape, bool)
    hit[2, 1] = hit[4, 2] = True
    assert np.isnan(s[hit]).all() and np.array_equal(s[~hit], s0[~hit])
    cols = hit[:, np.arange(384) // 128]
    assert np.all(q[cols] == 0x7F) and np.array_equal(q[~cols], q0[~cols])


def test_given_outputs_and_neighbours():
    x = torch.randn(9, 144).bfloat16()
    q = torch.full((11, 144), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((11, 2), -3.0, device="cuda")
    q2, s2 = fm.quant_fp8_blocks(x.cuda(), q=q[1:10], scale=s[1:10])
    torch.cuda.synchronize()
    assert q2.data_ptr() == q[1:].data_ptr() and s2.data_ptr() == s[1:].data_ptr()
    check(x, False, q2.cpu().numpy(), s2.cpu().numpy())
    assert torch.all(q[0] == 77) and torch.all(q[10] == 77) and torch.all(s[0] == -3) and torch.all(s[10] == -3)
