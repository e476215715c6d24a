"""The dense FP8 product and the ragged grouped products on the GPU against the float64 oracle.

Exact pins: operands are small whole numbers and scales powers of two, so that every partial sum is a whole multiple
of 1/4 below 2^22, which fp32 holds exactly in any order; fp32 outputs must be equal, bf16 outputs equal to the
rounded sum (halfway cases included).  A wrong row, column, block, scale or group shows there.

Random operands: FP8 sums are held to MFMA_REL_BOUND of the terms' magnitudes (the fp8 MFMA's own summation, measured
in gpu_helpers), bf16 sums to 2 K roundings of 2^-24 of them (any order of K additions, the products being exact);
bf16 outputs add half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle.products import block_product, ragged_product
from tests.gpu_helpers import MFMA_REL_BOUND, say

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
SENTINEL = -7.5
ROW, TILED = fm.WEIGHTS_ROW_MAJOR, fm.WEIGHTS_MFMA_TILED


def nb(n):
    return -(-n // 128)


def whole(g, shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=g).float()


def powers(g, shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g).float())


def operands(g, rows, N, K, E, fp8, exact):
    """(a, a_scale, b, b_scale) on the host; e4m3 or bf16."""
    t = E4M3 if fp8 else torch.bfloat16
    if exact:
        a, b = whole(g, (rows, K)), whole(g, (E, N, K))
        sa, sb = powers(g, (rows, nb(K))), powers(g, (E, nb(N), nb(K)))
    else:
        a, b = torch.randn(rows, K, generator=g) * 60, torch.randn(E, N, K, generator=g) * 60
        sa, sb = torch.rand(rows, nb(K), generator=g) * 0.02 + 1e-4, torch.rand(E, nb(N), nb(K), generator=g) * 2e-4
    a, b = a.clamp(-448, 448).to(t), b.clamp(-448, 448).to(t)
    return (a, sa, b, sb) if fp8 else (a, None, b, None)


def f64(t):
    return None if t is None else t.double().numpy()


def check(got, y, s, K, fp8, exact):
    """got (a host tensor) against sums y with term magnitudes s."""
    f32 = got.dtype == torch.float32
    if exact:
        want = torch.from_numpy(y).to(got.dtype)
        bad = torch.nonzero(got != want)
        assert not len(bad), f"{len(bad)} of {got.numel()} differ, first at {bad[0].tolist()}"
        return
    tol = s * (MFMA_REL_BOUND if fp8 else 2 * K * 2.0 ** -24)
    tol = tol + (0 if f32 else (np.abs(y) + tol) * 2.0 ** -8)
    err = np.abs(f64(got) - y)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance"


def gemm(a, sa, b, sb, layout=ROW, **kw):
    w = b.cuda()
    if layout == TILED:
        w = fm.pack_weights(w)
    out = fm.gemm_fp8_blocks(a.cuda(), sa.cuda(), w.view(torch.uint8)[0], sb[0].cuda(), weight_layout=layout, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def ragged(a, sa, b, sb, indptr, layout=ROW, out_dtype=torch.bfloat16):
    w = b.cuda()
    if layout == TILED:
        w = fm.pack_weights(w).view(b.dtype)
    ptr = torch.tensor(indptr, dtype=torch.int32).cuda()
    out = torch.full((a.shape[0], b.shape[1]), SENTINEL, dtype=out_dtype, device="cuda")
    if sa is None:
        fm.grouped_gemm_bf16_ragged(a.cuda(), w, ptr, out=out, weight_layout=layout)
    else:
        fm.grouped_gemm_fp8_ragged(a.cuda(), sa.cuda(), w, sb.cuda(), ptr, out=out, weight_layout=layout)
    torch.cuda.synchronize()
    return out.cpu()


# ---------------------------------------------------------------- dense

GEMM_SIZES = [(1, 1, 16), (1, 7168, 256), (2, 3, 48), (7, 130, 128), (15, 16, 144), (16, 31, 112), (17, 33, 400),
              (31, 128, 1024), (33, 257, 272), (64, 300, 256), (65, 64, 896), (100, 129, 640), (128, 256, 512),
              (129, 500, 1040), (200, 1000, 384), (257, 264, 784), (300, 520, 128), (513, 300, 1536), (700, 768, 656),
              (1030, 1100, 272), (2100, 260, 144)]


@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_exact(M, N, K, dtype):
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    ops = operands(g, M, N, K, 1, True, True)
    say("gemm exact", M, N, K, dtype)
    a, sa, b, sb = ops
    y, s = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    check(gemm(*ops, out_dtype=dtype), y, s, K, True, True)


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (5, 48, 256), (40, 272, 384), (130, 512, 1024), (300, 784, 640),
                                   (600, 256, 2048), (1500, 528, 128)])
def test_gemm_exact_tiled(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    a, sa, b, sb = ops = operands(g, M, N, K, 1, True, True)
    say("gemm exact tiled", M, N, K)
    y, s = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    check(gemm(*ops, layout=TILED, out_dtype=torch.float32), y, s, K, True, True)


@pytest.mark.parametrize("M,N,K", [(1, 500, 2048), (19, 70, 912), (150, 300, 1024), (520, 640, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_random(M, N, K, dtype):
    g = torch.Generator().manual_seed(M + 5 * N + K)
    a, sa, b, sb = ops = operands(g, M, N, K, 1, True, False)
    say("gemm random", M, N, K, dtype)
    y, s = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    check(gemm(*ops, out_dtype=dtype), y, s, K, True, False)


@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (21, 33, 272), (90, 300, 256), (300, 512, 640)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_addend(M, N, K, dtype):
    g = torch.Generator().manual_seed(M + N)
    a, sa, b, sb = ops = operands(g, M, N, K, 1, True, True)
    add = whole(g, (M, N), 100).to(torch.bfloat16)
    say("gemm addend", M, N, K, dtype)
    y, s = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    check(gemm(*ops, addend=add.cuda(), out_dtype=dtype), y + f64(add.float()), s, K, True, True)
    if dtype == torch.bfloat16:      # onto the addend itself
        out = add.cuda()
        got = gemm(*ops, addend=out, out=out)
        check(got, y + f64(add.float()), s, K, True, True)


@pytest.mark.parametrize("M", [3, 200])
def test_gemm_unaligned_out_and_row_slices(M):
    """out, addend and scales that start off 16-byte boundaries, a and b inside larger tensors."""
    g = torch.Generator().manual_seed(M)
    N, K = 44, 144
    a, sa, b, sb = operands(g, M + 1, N, K, 1, True, True)
    y, s = block_product(f64(a[1:].float()), f64(sa[1:]), f64(b[0].float()), f64(sb[0]))
    big = torch.full((M * N + 2,), SENTINEL, dtype=torch.bfloat16, device="cuda")
    out = big[1:-1].view(M, N)
    say("gemm unaligned", M)
    fm.gemm_fp8_blocks(a.cuda()[1:], sa.cuda()[1:], b.cuda()[0], sb.cuda()[0], out=out)
    torch.cuda.synchronize()
    check(out.cpu(), y, s, K, True, True)
    assert big[0].item() == SENTINEL and big[-1].item() == SENTINEL


@pytest.mark.parametrize("M,N,K", [(20, 40, 272), (300, 300, 272)])
def test_gemm_nan_and_inf_stay_in_their_rows_and_columns(M, N, K):
    g = torch.Generator().manual_seed(5)
    a, sa, b, sb = operands(g, M, N, K, 1, True, True)
    y, _ = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    a.view(torch.uint8)[M - 1, K - 1] = 0x7F
    b.view(torch.uint8)[0, N - 1, 130] = 0xFF
    sa[2, 1] = float("inf")
    say("gemm nan", M, N, K)
    got = gemm(a, sa, b, sb, out_dtype=torch.float32).double().numpy()
    bad = np.zeros((M, N), bool)
    bad[M - 1], bad[:, N - 1] = True, True
    assert np.isnan(got[bad]).all() and not np.isfinite(got[2]).any()
    bad[2] = True
    assert np.array_equal(got[~bad], y[~bad])


# ---------------------------------------------------------------- grouped

RAGGED = [
    # sizes of the groups, rows ahead of the first, rows behind the last, N, K (bytes of FP8; bf16 takes the same)
    ([1], 0, 0, 16, 16), ([0, 1, 0], 0, 2, 33, 48), ([3, 0, 17, 1], 1, 3, 40, 128), ([16, 16, 16], 0, 0, 64, 256),
    ([0, 0, 0], 0, 5, 32, 64), ([40, 1, 70, 0, 5], 2, 0, 130, 272), ([130, 260, 1], 0, 1, 300, 144),
    ([1] * 300, 0, 0, 48, 128), ([0] * 255 + [20, 3] + [0] * 300 + [50], 4, 4, 24, 80),
    ([600, 0, 333], 0, 7, 270, 384), ([2] * 1024, 1, 1, 16, 32), ([257] * 5, 0, 0, 256, 1024),
    ([1500], 10, 10, 600, 400), ([70, 65, 64, 63, 90, 33], 0, 0, 520, 640),
]


def ragged_case(sizes, before, after):
    indptr = np.concatenate([[0], np.cumsum(sizes)]) + before
    return indptr.tolist(), int(indptr[-1]) + after


@pytest.mark.parametrize("case", range(len(RAGGED)))
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ragged_exact(case, fp8, dtype):
    sizes, before, after, N, K = RAGGED[case]
    indptr, rows = ragged_case(sizes, before, after)
    g = torch.Generator().manual_seed(case)
    a, sa, b, sb = operands(g, rows, N, K, len(sizes), fp8, True)
    say("ragged exact", case, rows, N, K, fp8, dtype)
    got = ragged(a, sa, b, sb, indptr, out_dtype=dtype)
    y, s = ragged_product(f64(a.float()), f64(sa), f64(b.float()), f64(sb), indptr)
    inside = np.zeros(rows, bool)
    inside[indptr[0]:indptr[-1]] = True
    assert torch.all(got[~inside] == SENTINEL), "rows of no group were written"
    check(got[inside], y[inside], s[inside], K, fp8, True)


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 30], 48, 256), ([200, 1, 90], 272, 384), ([10] * 40, 64, 1024),
                                       ([700, 300], 528, 128)])
@pytest.mark.parametrize("fp8", [True, False])
def test_ragged_exact_tiled(sizes, N, K, fp8):
    indptr, rows = ragged_case(sizes, 1, 1)
    g = torch.Generator().manual_seed(N + K)
    a, sa, b, sb = operands(g, rows, N, K, len(sizes), fp8, True)
    say("ragged exact tiled", rows, N, K, fp8)
    got = ragged(a, sa, b, sb, indptr, TILED, torch.float32)
    y, s = ragged_product(f64(a.float()), f64(sa), f64(b.float()), f64(sb), indptr)
    assert torch.all(got[0] == SENTINEL) and torch.all(got[-1] == SENTINEL)
    check(got[1:-1], y[1:-1], s[1:-1], K, fp8, True)


@pytest.mark.parametrize("sizes,N,K", [([4, 0, 20, 2], 100, 784), ([300, 100], 260, 512)])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ragged_random(sizes, N, K, fp8, dtype):
    indptr, rows = ragged_case(sizes, 0, 0)
    g = torch.Generator().manual_seed(N + K)
    a, sa, b, sb = operands(g, rows, N, K, len(sizes), fp8, False)
    say("ragged random", rows, N, K, fp8, dtype)
    y, s = ragged_product(f64(a.float()), f64(sa), f64(b.float()), f64(sb), indptr)
    check(ragged(a, sa, b, sb, indptr, out_dtype=dtype), y, s, K, fp8, False)


@pytest.mark.parametrize("indptr,taken", [([0, 5, 3, 9], [(0, 0, 5), (2, 3, 9)]), ([-4, 6, 6, 40], [(0, 0, 6), (2, 6, 12)]),
                                          ([30, 50, 20, 12], [])])
def test_ragged_offsets_outside_the_rows(indptr, taken):
    """Offsets are cut to the rows, a group that ends ahead of its start is empty (overlapping groups get equal
    weights here, so their common rows have one value)."""
    g = torch.Generator().manual_seed(9)
    rows, N, K = 12, 40, 144
    a, sa, b, sb = operands(g, rows, N, K, 1, True, True)
    b, sb = b.repeat(3, 1, 1), sb.repeat(3, 1, 1)
    say("ragged offsets", indptr)
    got = ragged(a, sa, b, sb, indptr, out_dtype=torch.float32).double().numpy()
    y, _ = block_product(f64(a.float()), f64(sa), f64(b[0].float()), f64(sb[0]))
    want = np.full((rows, N), SENTINEL)
    for _, lo, hi in taken:
        want[lo:hi] = y[lo:hi]
    assert np.array_equal(got, want)


def test_products_are_deterministic():
    g = torch.Generator().manual_seed(11)
    a, sa, b, sb = operands(g, 300, 264, 912, 2, True, False)
    first = ragged(a, sa, b, sb, [0, 100, 300], out_dtype=torch.float32)
    assert torch.equal(first, ragged(a, sa, b, sb, [0, 100, 300], out_dtype=torch.float32))
    one = gemm(a, sa, b[:1], sb[:1], out_dtype=torch.float32)
    assert torch.equal(one, gemm(a, sa, b[:1], sb[:1], out_dtype=torch.float32))
