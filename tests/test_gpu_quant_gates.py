"""quant_fp8_blocks on the GPU, gated: values whose gate lies so far below zero that 1 / (1 + exp(-gate)) leaves the
normal range of fp32, while a large up brings the product back beside, or above, the other values of its block.

Tolerance: as for every other gate, (2 |g| + 8) 2^-24 relative, |g| taken as 90 at most (test_gpu_quant_blocks.check).
Below -87 the kernel takes 2^t with t = fma(g, -log2 e, -100): |t| < 128, so half a step of 2^-18, log2 e is off by
2^-25.4 relative, so |g| 2^-25.1 more, and ln 2 of both is at most 4.8e-6 for |g| <= 160; the exponential and the
reciprocal (2^-23 each) and two products (2^-24 each) add 3.6e-7.  5.2e-6 in all, below (2 * 87 + 8) 2^-24 = 1.08e-5.
"""

import numpy as np
import pytest
import torch

from oracle.products import silu_mul
from tests.gpu_helpers import say
from tests.test_gpu_quant_blocks import check, run

pytestmark = pytest.mark.gpu

GATES = [-80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -95.0, -100.0, -110.0, -130.0, -150.0]


def block(g, gates, ups, rest):
    """One row of 128 gates and ups, halves of a gated row: ordinary values whose products lie near `rest`, and the
    given ones at places drawn from g."""
    gate = torch.randn(128, generator=g, dtype=torch.float64) * 2
    up = torch.randn(128, generator=g, dtype=torch.float64) * rest
    at = torch.randperm(128, generator=g)[:len(gates)]
    gate[at], up[at] = torch.tensor(gates, dtype=torch.float64), torch.tensor(ups, dtype=torch.float64)
    return gate, up


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rest", [1.0, 1e-6, 1e-15, 1e10])
@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
def test_far_gates_beside_ordinary_values(dtype, rest, size):
    """Each far gate's up makes its value `size` times the others, as far as fp32 holds such an up."""
    g = torch.Generator().manual_seed(int(size * 7) + int(-np.log10(rest)) + 40)
    rows = []
    for i in range(len(GATES)):
        gates = [GATES[i], GATES[(i + 3) % len(GATES)], GATES[(i + 7) % len(GATES)]]
        ups = [np.clip(rest * size / (v / (1 + np.exp(-v))), -3e38, 3e38) for v in gates]
        rows.append(torch.cat(block(g, gates, ups, rest)))
    x = torch.stack(rows).to(dtype)
    say("far gates", dtype, rest, size)
    check(x, True, *run(x, True))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_far_gate_carries_its_block(dtype):
    """silu(-88) * 1e37 = -5.3 beside a block of at most 1e-3: the block's largest value."""
    x = torch.full((1, 256), 1e-3)
    x[0, 17], x[0, 128 + 17] = -88.0, 1e37
    x = x.to(dtype)
    q, s = run(x, True)
    check(x, True, q, s)
    v = silu_mul(x.double().numpy())
    assert v[0, 17] < -5 and q[0, 17] == 0xFE
