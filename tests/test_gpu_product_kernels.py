"""Every kernel that the products can take, in every layout and type, at sizes whose kernel is asserted first.

Whole-number operands and power-of-two scales make every sum exact (see test_gpu_products), so outputs are compared for
equality with the same product in float64.  Addends are whole numbers below 2^8, which bf16 holds; the sum is rounded
once.
"""

import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from tests.gpu_helpers import say
from tests.product_cases import DENSE, GROUPED, LARGEST, tiled_size
from tests.test_gpu_products_use import E4M3, gemm_operands, gen, nb, powers, product64, whole

pytestmark = pytest.mark.gpu

MARK = 99.0
LAYOUTS = [fm.WEIGHTS_ROW_MAJOR, fm.WEIGHTS_MFMA_TILED]


def plan_here(*size):
    return fm.product_plan(*size, num_cu=torch.cuda.get_device_properties(0).multi_processor_count)


def guarded(rows, N, dtype):
    """(a tensor with five marked rows behind the product's, the product's)."""
    t = torch.full((rows + 5, N), MARK, dtype=dtype, device="cuda")
    return t, t[:rows]


def dense(plan, M, N, K, layout):
    assert plan_here(M, N, K) == plan
    a, sa, b, sb = gemm_operands(gen(M + N + K), M, N, K)
    w = b if layout == fm.WEIGHTS_ROW_MAJOR else fm.pack_weights(b[None]).view(E4M3)[0]
    want = product64(a, sa, b, sb)
    add = whole(gen(M), M, N, dtype=torch.bfloat16, top=100)
    say("dense kernel", plan, M, N, K, layout)
    for dtype in (torch.float32, torch.bfloat16):
        for addend in (None, add):
            buf, out = guarded(M, N, dtype)
            fm.gemm_fp8_blocks(a, sa, w, sb, addend=addend, out=out, weight_layout=layout)
            exact = want if addend is None else want + add.double()
            assert torch.equal(out, exact.to(dtype)), (dtype, addend is not None)
            assert torch.all(buf[M:] == MARK)
    buf, out = guarded(M, N, torch.bfloat16)
    out.copy_(add)
    fm.gemm_fp8_blocks(a, sa, w, sb, addend=out, out=out, weight_layout=layout)
    assert torch.equal(out, (want + add.double()).to(torch.bfloat16)) and torch.all(buf[M:] == MARK)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("plan", DENSE, ids=str)
def test_dense_kernels(plan, layout):
    dense(plan, *DENSE[plan][layout], layout)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("pair", LARGEST, ids=str)
def test_largest_dense_tile(pair, layout):
    dense((256, 256, 8, 1), *pair[layout], layout)


def uneven(g, rows, E):
    """Sizes of E groups that add up to rows, some empty where there are several."""
    p = torch.rand(E, generator=g, device="cuda") + 0.5
    if E > 2:
        p[1::4] = 0
    group = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(group, minlength=E)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("plan", GROUPED, ids=str)
def test_grouped_kernels(plan, bf16, layout):
    rows, N, K, E = GROUPED[plan][bf16]
    if layout == fm.WEIGHTS_MFMA_TILED:
        N, K = tiled_size(N, K, bf16)
    assert plan_here(rows, N, K, E, bf16) == plan
    g = gen(rows + N + K + E)
    sizes = uneven(g, rows - 4, E)
    ptr = torch.cat([torch.tensor([1], device="cuda"), sizes.cumsum(0) + 1]).to(torch.int32)
    t = torch.bfloat16 if bf16 else E4M3
    a, b = whole(g, rows, K, dtype=t), whole(g, E, N, K, dtype=t)
    sa = sb = None
    if not bf16:
        sa, sb = powers(g, rows, nb(K)), powers(g, E, nb(N), nb(K))
    w = b if layout == fm.WEIGHTS_ROW_MAJOR else fm.pack_weights(b).view(t)
    want = torch.full((rows, N), MARK, dtype=torch.float64, device="cuda")
    ends = ptr.tolist()
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        want[r] = product64(a[r], None if bf16 else sa[r], b[e], None if bf16 else sb[e])
    say("grouped kernel", plan, bf16, layout, rows, N, K, E)
    for dtype in (torch.float32, torch.bfloat16):
        buf, out = guarded(rows, N, dtype)
        if bf16:
            fm.grouped_gemm_bf16_ragged(a, w, ptr, out=out, weight_layout=layout)
        else:
            fm.grouped_gemm_fp8_ragged(a, sa, w, sb, ptr, out=out, weight_layout=layout)
        assert torch.equal(out, want.to(dtype)), dtype       # rows of no group keep their mark
        assert torch.all(buf[rows:] == MARK)
