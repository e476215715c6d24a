"""The choice of the products' kernels, without a GPU: which kernel each size of the GPU tests takes, and that those
sizes reach every kernel and number of parts that the choice can give."""

import ctypes
import math
import random

import pytest

import fp8_block_scaled_moe_amd as fm
from fp8_block_scaled_moe_amd._lib import lib
from tests.product_cases import DENSE, GROUPED, LARGEST, tiled_size


@pytest.mark.parametrize("plan", DENSE, ids=str)
def test_dense_sizes_take_their_kernels(plan):
    for M, N, K in DENSE[plan]:
        assert fm.product_plan(M, N, K) == plan, (M, N, K)
    assert DENSE[plan][0][2] % 128 and DENSE[plan][1][1] % 16 == 0 and DENSE[plan][1][2] % 128 == 0


def test_more_of_the_largest_tile():
    for pair in LARGEST:
        for M, N, K in pair:
            assert fm.product_plan(M, N, K) == (256, 256, 8, 1), (M, N, K)


@pytest.mark.parametrize("plan", GROUPED, ids=str)
@pytest.mark.parametrize("bf16", [False, True])
def test_grouped_sizes_take_their_kernels(plan, bf16):
    rows, N, K, E = GROUPED[plan][bf16]
    assert K * (2 if bf16 else 1) % 128
    assert fm.product_plan(rows, N, K, E, bf16) == plan
    assert fm.product_plan(rows, *tiled_size(N, K, bf16), E, bf16) == plan


def test_no_other_kernel_is_taken():
    r = random.Random(1)

    def log(lo, hi):
        return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))

    for _ in range(40000):
        size = log(1, 1 << 20), log(1, 65536), 16 * log(1, 4096)
        assert fm.product_plan(*size) in DENSE, size
        size = log(1, 1 << 20), log(1, 65536), 16 * log(1, 4096), log(1, 1024), r.random() < 0.5
        assert fm.product_plan(*size) in GROUPED, size
    for size in (((1 << 30) - 1, 65536, 65536), ((1 << 30) - 1, 1, 16), (1, 65536, 65536), (1, 1, 16)):
        assert fm.product_plan(*size) in DENSE
        for E in (1, 1024):
            assert fm.product_plan(*size, E, True) in GROUPED


def test_parts_fit_the_workspace():
    r = random.Random(2)
    for _ in range(20000):
        M, N, K = r.randint(1, 3000), r.randint(1, 9000), 16 * r.randint(1, 1200)
        parts = fm.product_plan(M, N, K)[3]
        if parts > 1:
            assert 4 * parts * M * ((N + 7) // 8 * 8) <= fm.gemm_workspace_size(M, N, K)
            assert -(-K // 128) >= 8 * parts


def test_plan_refusals():
    v = [ctypes.c_int32(7) for _ in range(4)]
    p = [ctypes.byref(x) for x in v]
    call = lib().moe_product_plan
    assert call(1, 16, 16, 0, 0, 256, *p) == 0
    for args, status in (((0, 16, 16, 0, 0, 256), -2), ((-1, 16, 16, 0, 0, 256), -2), ((1, 0, 16, 0, 0, 256), -2),
                         ((1, 16, 0, 0, 0, 256), -2), ((1, 16, 16, -1, 0, 256), -2), ((1, 16, 16, 0, 1, 256), -2),
                         ((1, 16, 16, 0, 0, 0), -2), ((1, 16, 24, 0, 0, 256), -3), ((1, 16, 12, 1, 1, 256), -3),
                         ((1 << 30, 16, 16, 0, 0, 256), -8), ((1, 65537, 16, 0, 0, 256), -8),
                         ((1, 16, 65552, 1, 0, 256), -8), ((1, 16, 16, 1025, 0, 256), -8)):
        assert call(*args, *p) == status, args
    for i in range(4):
        assert call(1, 16, 16, 0, 0, 256, *[None if k == i else p[k] for k in range(4)]) == -1
    with pytest.raises(fm.Fp8MoeError):
        fm.product_plan(0, 16, 16)
