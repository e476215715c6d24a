"""The norm's eps: refused where fp32 holds it, or its sum with a mean square, badly.  No GPU is touched."""

import ctypes

import pytest

import fp8_block_scaled_moe_amd as fm
from fp8_block_scaled_moe_amd._lib import lib

NULL = ctypes.c_void_p(0)


@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-40, 2.0 ** -127, 2.0 ** 127, 3.4e38])
def test_eps_outside_its_range(eps):
    p = [ctypes.c_void_p((i + 1) << 34) for i in range(4)]
    args = (p[0], NULL, 0, p[1], 0)
    out = (256, fm.NORM_INT8, NULL, NULL, p[2], p[3], NULL)
    assert lib().add_rmsnorm_quant(*args, eps, 0, *out) == -9
    assert b"eps" in lib().moe_last_error()
    for good in (2.0 ** -126, 1e-6, 2.0 ** 126):
        assert lib().add_rmsnorm_quant(*args, good, 0, *out) == 0
