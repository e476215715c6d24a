"""Host-side checks of the products' and the block quantiser's entry points: invalid arguments are refused before
any launch, and empty calls succeed."""

import ctypes

import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from fp8_block_scaled_moe_amd._lib import lib

OK, E_NULL, E_SHAPE, E_ALIGN, E_WS, E_LIMIT = 0, -1, -2, -3, -6, -8
NULL = ctypes.c_void_p(0)


def P(i, off=0):
    """Device pointers 64 GiB apart, never dereferenced: every call below fails validation first."""
    return ctypes.c_void_p(((i + 1) << 36) + off)


def gemm(a=P(0), sa=P(1), b=P(2), sb=P(3), add=NULL, M=4, N=24, K=256, out=P(4), f32=0, ws=P(5), wsb=1 << 34, layout=0):
    return lib().gemm_fp8_blocks(a, sa, b, sb, add, M, N, K, out, f32, ws, wsb, layout, NULL)


def ragged8(a=P(0), sa=P(1), b=P(2), sb=P(3), ptr=P(5), rows=4, N=24, K=256, E=3, out=P(4), f32=0, layout=0):
    return lib().moe_grouped_gemm_fp8_ragged(a, sa, b, sb, ptr, rows, N, K, E, out, f32, layout, NULL)


def ragged16(a=P(0), b=P(2), ptr=P(5), rows=4, N=24, K=256, E=3, out=P(4), f32=0, layout=0):
    return lib().moe_grouped_gemm_bf16_ragged(a, b, ptr, rows, N, K, E, out, f32, layout, NULL)


def quant(x=P(0), f32=0, M=4, N=256, gated=0, q=P(1), s=P(2)):
    return lib().quant_fp8_blocks(x, f32, M, N, gated, q, s, NULL)


@pytest.mark.parametrize("call,rows", [(gemm, "M"), (ragged8, "rows"), (ragged16, "rows")])
def test_product_sizes(call, rows):
    assert call(**{rows: -1}) == E_SHAPE and call(N=0) == E_SHAPE and call(K=0) == E_SHAPE and call(K=-16) == E_SHAPE
    assert call(**{rows: 1 << 30}) == E_LIMIT and call(N=65537) == E_LIMIT and call(K=65536 + 16) == E_LIMIT
    assert call(layout=2) == E_SHAPE and call(layout=-1) == E_SHAPE
    assert call(K=260) == E_ALIGN
    assert call(layout=1) == E_ALIGN                       # N = 24
    assert call(layout=1, N=32, K=200 if call is ragged16 else 144) == E_ALIGN
    assert call(**{rows: 0}, a=NULL, b=NULL, out=NULL) == OK


@pytest.mark.parametrize("call", [ragged8, ragged16])
def test_ragged_groups(call):
    assert call(E=0) == E_SHAPE and call(E=1025) == E_LIMIT
    assert call(ptr=NULL) == E_NULL and call(ptr=P(5, 2)) == E_ALIGN
    assert call(out=P(5)) == E_SHAPE                       # over m_indptr


@pytest.mark.parametrize("call", [gemm, ragged8, ragged16])
def test_product_tensors(call):
    assert call(a=NULL) == E_NULL and call(b=NULL) == E_NULL and call(out=NULL) == E_NULL
    assert call(a=P(0, 8)) == E_ALIGN and call(b=P(2, 4)) == E_ALIGN
    assert call(out=P(4, 1)) == E_ALIGN and call(out=P(4, 2), f32=1) == E_ALIGN
    assert call(out=P(0)) == E_SHAPE and call(out=P(2, 16)) == E_SHAPE
    assert call(out=P(0, -16)) == E_SHAPE                  # its end reaches into a
    if call is not ragged16:
        assert call(sa=NULL) == E_NULL and call(sb=NULL) == E_NULL
        assert call(sa=P(1, 2)) == E_ALIGN and call(sb=P(3, 1)) == E_ALIGN
        assert call(out=P(1)) == E_SHAPE and call(out=P(3)) == E_SHAPE


def test_gemm_addend():
    assert gemm(add=P(6, 1)) == E_ALIGN
    assert gemm(add=P(4, 16)) == E_SHAPE                   # out shifted over its own addend
    assert gemm(add=P(4), f32=1) == E_SHAPE                # of another type than out


def test_gemm_workspace_size():
    n = ctypes.c_size_t(7)
    assert lib().gemm_fp8_blocks_workspace_size(4, 24, 256, ctypes.byref(n)) == OK
    assert lib().gemm_fp8_blocks_workspace_size(4, 24, 256, None) == E_NULL
    assert lib().gemm_fp8_blocks_workspace_size(-1, 24, 256, ctypes.byref(n)) == E_SHAPE
    assert lib().gemm_fp8_blocks_workspace_size(4, 24, 250, ctypes.byref(n)) == E_ALIGN
    assert fm.gemm_workspace_size(0, 24, 256) >= 0


def test_quant_validation():
    assert quant(M=-1) == E_SHAPE and quant(N=0) == E_SHAPE
    assert quant(N=24) == E_ALIGN and quant(N=8) == E_ALIGN
    assert quant(N=65536 + 16) == E_LIMIT and quant(M=1 << 30) == E_LIMIT
    assert quant(x=NULL) == E_NULL and quant(q=NULL) == E_NULL and quant(s=NULL) == E_NULL
    assert quant(x=P(0, 8)) == E_ALIGN and quant(q=P(1, 8)) == E_ALIGN and quant(s=P(2, 2)) == E_ALIGN
    assert quant(q=P(0)) == E_SHAPE and quant(s=P(0)) == E_SHAPE and quant(q=P(2)) == E_SHAPE
    assert quant(q=P(0, 4 * 256 * 4 - 16), f32=1) == E_SHAPE
    assert quant(q=P(0, 4 * 512 * 2 - 16), gated=1) == E_SHAPE
    assert quant(M=0, x=NULL, q=NULL, s=NULL) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    a, s = torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4, 1)
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, s, a, s)
    with pytest.raises(TypeError):
        fm.gemm_fp8_blocks(a.int(), s, a, s)
    with pytest.raises(TypeError):
        fm.gemm_fp8_blocks(None, s, a, s)
    with pytest.raises(TypeError):
        fm.grouped_gemm_bf16_ragged(a, a, a)
    with pytest.raises(ValueError):
        fm.quant_fp8_blocks(torch.zeros(4, 128))
    with pytest.raises(TypeError):
        fm.quant_fp8_blocks(torch.zeros(4, 128, dtype=torch.float16))


def test_gemm_workspace_serves_smaller_batches():
    """The size never falls as M grows and stays bounded; calls refuse a smaller, missing or unaligned one."""
    for N, K in ((576, 7168), (7168, 2048), (1, 65536), (65536, 128)):
        sizes = [fm.gemm_workspace_size(M, N, K) for M in (0, 1, 2, 16, 33, 64, 200, 1000, 5000, 100000, (1 << 30) - 1)]
        assert sizes == sorted(sizes) and sizes[-1] <= 16 << 20
    need = fm.gemm_workspace_size(4, 24, 2048)
    assert need > 0 and need % 256 == 0
    assert gemm(K=2048, ws=NULL) == E_WS and gemm(K=2048, wsb=need - 1) == E_WS and gemm(K=2048, ws=P(5, 128)) == E_WS
    assert gemm(K=2048, ws=P(0)) == E_SHAPE and gemm(K=2048, ws=P(4)) == E_SHAPE and gemm(K=2048, add=P(5)) == E_SHAPE
