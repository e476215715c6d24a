"""Host-side checks of the norm's, the router's and the int8 layer's entry points: invalid arguments are refused
before any launch, empty calls succeed, and the oracles agree with brute force."""

import ctypes

import numpy as np
import pytest

import fp8_block_scaled_moe_amd as fm
from fp8_block_scaled_moe_amd._lib import lib
from oracle import int8 as O8
from oracle.norm import add_rmsnorm_reference
from oracle.router import router_reference

OK, E_NULL, E_SHAPE, E_ALIGN, E_TOPK, E_TILE, E_WS, E_LIMIT, E_ARG = 0, -1, -2, -3, -4, -5, -6, -8, -9
NULL = ctypes.c_void_p(0)


def P(i):
    """Device pointers 16 GiB apart, never dereferenced: every call below fails validation first."""
    return ctypes.c_void_p((i + 1) << 34)


def norm(x=P(0), res=P(1), r32=0, w=P(2), w32=0, eps=1e-6, T=4, H=256, fmt=fm.NORM_FP8, res_out=P(3), norm_out=P(4),
         q=P(5), scale=P(6)):
    return lib().add_rmsnorm_quant(x, res, r32, w, w32, eps, T, H, fmt, res_out, norm_out, q, scale, NULL)


def test_norm_validation():
    assert norm(T=-1) == E_SHAPE
    assert norm(H=0) == E_SHAPE
    for fmt, H in ((fm.NORM_FP8, 192), (fm.NORM_MXFP8, 48), (fm.NORM_INT8, 12), (fm.NORM_BF16, 4)):
        assert norm(fmt=fmt, H=H) == E_ALIGN
    assert norm(H=16384 + 128) == E_LIMIT
    assert norm(T=1 << 24) == E_LIMIT
    assert norm(fmt=4) == E_ARG and norm(fmt=-1) == E_ARG
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == E_ARG
    assert norm(res=NULL) == E_NULL and norm(res_out=NULL) == E_NULL
    assert norm(x=NULL) == E_NULL and norm(w=NULL) == E_NULL and norm(q=NULL) == E_NULL and norm(scale=NULL) == E_NULL
    assert norm(fmt=fm.NORM_BF16, norm_out=NULL) == E_NULL
    off = ctypes.c_void_p((9 << 34) + 8)
    for k in ("x", "w", "norm_out", "q", "scale"):
        assert norm(**{k: off}) == E_ALIGN
    assert norm(res=off) == E_ALIGN and norm(res_out=off) == E_ALIGN
    assert norm(q=P(0)) == E_SHAPE and norm(norm_out=P(1)) == E_SHAPE and norm(scale=P(5)) == E_SHAPE
    assert norm(res_out=ctypes.c_void_p((2 << 34) + 16)) == E_SHAPE        # shifted over its own input
    assert norm(q=ctypes.c_void_p((1 << 34) + 4 * 256 * 2 - 16)) == E_SHAPE
    assert norm(T=0, x=NULL, res=NULL, w=NULL, res_out=NULL, norm_out=NULL, q=NULL, scale=NULL) == OK
    assert lib().moe_status_string(E_ARG).decode() != "unknown status"


def router(logits=P(0), bf16=0, bias=P(1), T=4, E=64, K=4, score=0, n_group=1, topk_group=1, group_top=1, renorm=1,
           scale=1.0, ids=P(2), w=P(3)):
    return lib().moe_router_topk(logits, bf16, bias, T, E, K, score, n_group, topk_group, group_top, renorm, scale,
                                 ids, w, NULL)


def test_router_validation():
    assert router(T=-1) == E_SHAPE and router(E=0) == E_SHAPE
    assert router(E=1025) == E_LIMIT and router(T=1 << 25) == E_LIMIT
    assert router(K=0) == E_TOPK and router(K=65) == E_TOPK and router(K=5, E=4) == E_TOPK
    assert router(K=17, n_group=4, topk_group=1) == E_TOPK
    assert router(score=2) == E_ARG and router(score=-1) == E_ARG
    assert router(n_group=0) == E_ARG and router(n_group=5) == E_ARG and router(n_group=128, E=256) == E_ARG
    assert router(n_group=4, topk_group=5) == E_ARG and router(n_group=4, topk_group=0) == E_ARG
    assert router(group_top=0) == E_ARG and router(group_top=3) == E_ARG
    assert router(n_group=64, topk_group=4, group_top=2) == E_ARG
    assert router(scale=float("nan")) == E_ARG and router(scale=float("inf")) == E_ARG
    for k in ("logits", "ids", "w"):
        assert router(**{k: NULL}) == E_NULL
    assert router(ids=P(0)) == E_SHAPE and router(w=P(1)) == E_SHAPE and router(w=P(2)) == E_SHAPE
    assert router(w=ctypes.c_void_p((3 << 34) + 4 * 4 * 4 - 4)) == E_SHAPE
    assert router(T=0, logits=NULL, bias=NULL, ids=NULL, w=NULL) == OK


def fused(T=16, H=256, I=128, E=4, K=2, ptr=P(0), ws=P(1), wsb=1 << 40, tm=-1, out=P(2), layout=0):
    return lib().moe_fused_int8(ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, T, H, I, E, K, out, ws, wsb, tm, layout, NULL)


def test_int8_validation():
    assert fused(T=-1) == E_SHAPE and fused(H=0) == E_SHAPE and fused(E=0) == E_SHAPE
    assert fused(H=200) == E_ALIGN and fused(I=100) == E_ALIGN
    assert fused(K=5) == E_TOPK and fused(K=0) == E_TOPK
    assert fused(E=1025) == E_LIMIT and fused(H=16384 + 128) == E_LIMIT
    assert fused(tm=48) == E_TILE and fused(tm=512) == E_TILE
    assert fused(layout=2) == E_SHAPE
    assert fused(ptr=NULL) == E_NULL and fused(out=NULL) == E_NULL
    assert fused(ptr=ctypes.c_void_p((1 << 34) + 8)) == E_ALIGN
    assert fused(ws=NULL) == E_WS and fused(wsb=1024) == E_WS and fused(ws=ctypes.c_void_p(0x1010)) == E_WS
    assert fused(T=0, ptr=NULL, ws=NULL, out=NULL) == OK
    p, odd = P(0), ctypes.c_void_p((1 << 34) + 4)
    for scales in ((odd, p), (p, odd)):
        assert lib().moe_fused_int8(p, p, p, scales[0], p, scales[1], p, p, 16, 256, 128, 4, 2, P(2), P(1), 1 << 40, -1,
                                    0, NULL) == E_ALIGN
    n = fm.fused_int8_workspace_size(16, 256, 128, 4, 2)
    cap, R = 32 + 4 * 15, 32
    assert n >= cap * 128 * 3 + cap * 8 + R * 256 * 2
    with pytest.raises(fm.Fp8MoeError):
        fm.fused_int8_workspace_size(16, 200, 128, 4, 2)


def test_int8_stage_validation():
    L, a, s = lib(), P(0), P(1)

    def gemm1(T=4, H=256, I=128, E=4, K=2, align=16, cap=68, tm=-1, layout=0, p=a):
        return L.moe_gemm1_swiglu_int8(p, s, p, s, s, s, T, H, I, E, K, align, p, cap, tm, layout, NULL)

    def gemm2(T=4, H=256, I=128, E=4, K=2, align=16, cap=68, tm=-1, layout=0, p=a):
        return L.moe_gemm2_weighted_int8(p, s, p, s, s, s, s, T, H, I, E, K, align, p, cap, tm, layout, NULL)

    for f in (gemm1, gemm2):
        assert f(H=100) == E_ALIGN and f(align=48) == E_ALIGN and f(K=5) == E_TOPK and f(tm=20) == E_TILE
        assert f(cap=-1) == E_SHAPE and f(layout=3) == E_SHAPE and f(p=NULL) == E_NULL
        assert f(p=ctypes.c_void_p((1 << 34) + 4)) == E_ALIGN
        assert f(T=0, p=NULL) == OK and f(cap=0, p=NULL) == OK

    def rows(inp=a, rows=4, N=64, q=P(2), scale=P(3)):
        return L.moe_quant_rows_int8(inp, NULL, rows, N, q, scale, NULL)

    assert rows(rows=-1) == E_SHAPE and rows(N=0) == E_SHAPE and rows(N=12) == E_ALIGN
    assert rows(inp=NULL) == E_NULL and rows(q=NULL) == E_NULL and rows(scale=NULL) == E_NULL
    assert rows(q=a) == E_SHAPE and rows(q=ctypes.c_void_p((3 << 34) + 8)) == E_ALIGN
    assert rows(rows=0, inp=NULL, q=NULL, scale=NULL) == OK


def test_oracle_norm():
    v, n = add_rmsnorm_reference([[3.0, 4.0]], None, [1.0, 2.0], 1e-12, False)
    assert np.allclose(n, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-12)
    v, _ = add_rmsnorm_reference([[1.0]], [[2.0 ** -9]], [1.0], 1e-6, True)      # lost in bf16
    assert v[0, 0] == 1.0


def test_oracle_router():
    x = [[0.0, 2.0, 1.0, 2.0]]
    ids, w = router_reference(x, 2, "softmax")
    assert ids.tolist() == [[1, 3]] and np.allclose(w, 0.5)
    ids, w = router_reference(x, 2, "softmax", n_group=2, topk_group=1)            # both groups' best is 2
    assert ids.tolist() == [[1, 0]]
    ids, w = router_reference(x, 2, "sigmoid", bias=[0, 0, 1.0, 0], renormalize=False, scale=2.0)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, 2 / (1 + np.exp([[-1.0, -2.0]])))
    ids, w = router_reference([[-np.inf, np.nan, 0.0]], 2, "sigmoid")
    assert ids.tolist() == [[2, -1]] and w[0, 1] == 0


def test_oracle_int8():
    rng = np.random.default_rng(0)
    x, w = rng.integers(-127, 128, (3, 8)), rng.integers(-127, 128, (4, 8))
    xs, ws = rng.random(3), rng.random(4)
    h = O8.int8_product(x, xs, w, ws)
    for i in range(3):
        for j in range(4):
            assert np.isclose(h[i, j], sum(int(a) * int(b) for a, b in zip(x[i], w[j])) * xs[i] * ws[j], rtol=1e-14)
    q, s = O8.quantize_rows_int8([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0]])
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0]] and s.tolist() == [1.0, 1.0]
