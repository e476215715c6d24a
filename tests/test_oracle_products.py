"""Pins of oracle/products.py: scalar brute force, closed forms, and invariants."""

import numpy as np

from oracle.products import block_product, quant_blocks, ragged_product, silu_mul


def test_block_product_brute_force():
    r = np.random.default_rng(1)
    M, N, K = 3, 131, 140
    a, b = r.integers(-3, 4, (M, K)), r.integers(-3, 4, (N, K))
    sa, sb = r.random((M, 2)), r.random((2, 2))
    y, s = block_product(a, sa, b, sb)
    for m in range(M):
        for n in (0, 1, 127, 128, 130):
            t = [a[m, k] * sa[m, k // 128] * b[n, k] * sb[n // 128, k // 128] for k in range(K)]
            assert abs(y[m, n] - sum(t)) < 1e-9 and abs(s[m, n] - sum(map(abs, t))) < 1e-9


def test_block_product_unit_scales_and_single_blocks():
    r = np.random.default_rng(2)
    a, b = r.standard_normal((4, 256)), r.standard_normal((200, 256))
    one = block_product(a, np.ones((4, 2)), b, np.ones((2, 2)))[0]
    assert np.allclose(one, a @ b.T) and np.allclose(one, block_product(a, None, b, None)[0])
    sb = np.zeros((2, 2))
    sb[1, 0] = 2.0
    y = block_product(a, np.ones((4, 2)), b, sb)[0]
    assert np.all(y[:, :128] == 0) and np.allclose(y[:, 128:], 2 * a[:, :128] @ b[128:, :128].T)


def test_ragged_product_groups():
    r = np.random.default_rng(3)
    a, b = r.standard_normal((10, 32)), r.standard_normal((4, 5, 32))
    y, _ = ragged_product(a, None, b, None, [1, 4, 4, 9, 9])
    assert np.isnan(y[0]).all() and np.isnan(y[9]).all()
    for m in range(1, 9):
        assert np.allclose(y[m], b[0 if m < 4 else 2] @ a[m])


def test_quant_blocks_invariants():
    r = np.random.default_rng(4)
    v = r.standard_normal((5, 300))
    v[2, 128:256] = 0
    q, s = quant_blocks(v)
    assert s.shape == (5, 3) and s[2, 1] == 1 and np.all(q[2, 128:256] == 0)
    for k in range(3):
        top = np.abs(q[:, 128 * k:128 * k + 128]).max(1)
        assert np.allclose(np.delete(top, 2) if k == 1 else top, 448)
    assert np.allclose(q * s[:, np.arange(300) // 128], v)


def test_silu_mul_closed_forms():
    assert np.all(silu_mul([[0.0, 3.0]]) == 0)
    assert np.allclose(silu_mul([[2.0, 3.0]]) - silu_mul([[-2.0, 3.0]]), 6.0)
    assert silu_mul([[-1000.0, 1.0]])[0, 0] == 0 and silu_mul([[1000.0, 2.0]])[0, 0] == 2000
