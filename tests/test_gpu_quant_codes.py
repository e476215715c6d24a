"""quant_fp8_blocks on the GPU, ungated: codes and scales equal to the definition evaluated in fp32 on the host, scale =
amax / 448 by IEEE division and q = e4m3 of the correctly rounded fp32 quotient, ties to even.  No tolerance: a quotient
that is an ulp off moves a code wherever it lies on the middle of two, which bf16 values meet often.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def fp32_definition(x):
    """(codes, scales) of fp32 x [M, N]: numpy divides in fp32 by IEEE, torch rounds to e4m3 to nearest even."""
    M, N = x.shape
    v = x.numpy()
    codes, scale = np.empty((M, N), np.uint8), np.empty((M, -(-N // 128)), np.float32)
    for k in range(scale.shape[1]):
        c = slice(128 * k, min(128 * k + 128, N))
        s = np.abs(v[:, c]).max(1) / np.float32(448)
        scale[:, k] = np.where(s > 0, s, np.float32(1))
        q = np.clip(v[:, c] / scale[:, k, None], np.float32(-448), np.float32(448))
        codes[:, c] = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, scale


def compare(x):
    q, s = fm.quant_fp8_blocks(x.cuda())
    torch.cuda.synchronize()
    want_q, want_s = fp32_definition(x.float())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    bad = np.argwhere(q.cpu().numpy() != want_q)
    assert not len(bad), f"{len(bad)} of {want_q.size} codes differ, first at {bad[0].tolist()}"


@pytest.mark.parametrize("M,N", [(1, 16), (1, 7168), (37, 400), (2000, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_are_those_of_the_rounded_quotient(M, N, dtype):
    g = torch.Generator().manual_seed(M + N)
    say("codes", M, N, dtype)
    compare((torch.randn(M, N, generator=g) * (1 + 20 * (torch.rand(N, generator=g) < 0.01))).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_of_every_size(dtype):
    """Blocks from fp32's smallest numbers to its largest, the scale's underflow among them."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3000, 256, generator=g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-148, 126, (3000, 2), generator=g).double()).repeat_interleave(128, 1)
    say("codes of every size", dtype)
    compare(x.clamp(-3e38, 3e38).float().to(dtype))


def middles():
    """Each positive middle of two neighbouring e4m3 values up to 448 (and half the smallest)."""
    v = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("amax", [448.0, 1.0, 416.0, 2.0 ** -30, 240.0, 3.390625, 255.0])
def test_middles_of_codes(amax):
    """Every middle of two codes, times the scale, rounded to fp32 and to bf16, and the values beside them."""
    mid = middles()
    say("middles", amax)
    scale = float(np.float32(amax) / np.float32(448))
    for dtype, step in ((torch.float32, 2.0 ** -23), (torch.bfloat16, 2.0 ** -7)):
        near = torch.stack([(mid * scale * (1 + d * step)).to(dtype) for d in (-1, 0, 1)])
        rows = torch.zeros(6, 128, dtype=dtype)
        rows[:3, :126], rows[3:, :126] = near, -near
        rows[:, 127] = amax
        rows[:, :126] = torch.where(rows[:, :126].abs() <= amax, rows[:, :126], torch.zeros((), dtype=dtype))
        compare(rows)


@pytest.mark.parametrize("gated", [False, True])
def test_codes_into_a_float8_tensor(gated):
    """q of the type that the products take as a: the same codes, into the caller's tensor."""
    x = torch.randn(9, 288, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    want, scale = fm.quant_fp8_blocks(x, gated=gated)
    q = torch.zeros(want.shape, dtype=torch.float8_e4m3fn, device="cuda")
    got, s = fm.quant_fp8_blocks(x, gated=gated, q=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q.view(torch.uint8), want) and torch.equal(s, scale)
    for bad in (torch.int8, torch.float8_e5m2):
        with pytest.raises(TypeError):
            fm.quant_fp8_blocks(x, gated=gated, q=torch.zeros(want.shape, dtype=bad, device="cuda"))
