"""add_rmsnorm_quant over many rows, where a row has fewer threads than vectors, against the float64 oracle.

Tolerances.  v is exact.  A thread sums at most 64 squares and at most 16 waves' sums meet, after 6 steps inside a
wave: the mean square, of positive terms, is within 86 * 2^-24 relative; halved by the root, plus mean, eps, root,
reciprocal and the two products: n is within DELTA = 50 * 2^-24 relative.  Codes are held to the rounding interval of
n / scale for the scale the GPU stored.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle.norm import add_rmsnorm_reference
from tests.gpu_helpers import e4m3_rounding_interval, e8m0_exponent_range, say

pytestmark = pytest.mark.gpu

DELTA = 50 * 2.0 ** -24
FORMATS = {"bf16": fm.NORM_BF16, "fp8": fm.NORM_FP8, "mxfp8": fm.NORM_MXFP8, "int8": fm.NORM_INT8}
INF, NAN = float("inf"), float("nan")


def make(T, H, residual="bf16", weight="bf16", seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).bfloat16()
    r = None if residual == "none" else torch.randn(T, H, generator=g) * 3
    r = r.bfloat16() if residual == "bf16" else r
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x, r, (w.bfloat16() if weight == "bf16" else w)


def run(x, r, w, eps, fmt, **kw):
    c = lambda t: None if t is None else t.cuda()
    out = fm.add_rmsnorm_quant(c(x), c(w), eps, FORMATS[fmt], residual=c(r), want_norm=True, **kw)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in out]


def f64(t):
    return None if t is None else t.double().numpy()


def check(x, r, w, eps, fmt, out):
    """Every finite row of out = (q, scale, norm, v) against the oracle."""
    q, scale, norm, v = out
    T, H = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        vr, n = add_rmsnorm_reference(f64(x), f64(r), f64(w), eps, r is not None and r.dtype == torch.bfloat16)
    if r is not None:
        assert np.array_equal(f64(v), vr, equal_nan=True)
    ok = np.isfinite(vr).all(1)
    n, bad = n[ok], torch.from_numpy(~ok)
    assert torch.isnan(norm[bad]).all()
    assert np.all(np.abs(f64(norm)[ok] - n) <= np.abs(n) * (2.0 ** -8 + 2 * DELTA) + 2.0 ** -133)
    if fmt == "bf16":
        assert q is None and scale is None
        return
    if fmt == "int8":
        assert torch.isnan(scale[bad]).all() and not q[bad].any()
        amax = np.abs(n).max(1)
        want = np.where(amax > 0, amax / 127, 1.0)
        assert np.all(np.abs(f64(scale)[ok] - want) <= want * (DELTA + 2.0 ** -23))
        exact = n / f64(scale)[ok][:, None]
        assert np.all(np.abs(f64(q)[ok] - exact) <= 0.5 + np.abs(exact) * 2 * DELTA)
        return
    assert (q[bad] == 0x7F).all()
    if fmt == "fp8":
        assert torch.isnan(scale[bad]).all()
        amax = np.abs(n).reshape(len(n), -1, 128).max(2)
        want = np.where(amax > 0, amax / 448, 1.0)
        assert np.all(np.abs(f64(scale)[ok] - want) <= want * (DELTA + 2.0 ** -23))
        s = f64(scale)[ok].repeat(128, 1)
    else:
        assert (scale[bad] == 255).all()
        amax = np.abs(n).reshape(len(n), -1, 32).max(2)
        lo, hi = e8m0_exponent_range(amax * (1 - DELTA), amax * (1 + DELTA))
        e = scale.numpy()[ok].astype(np.int64) - 127
        assert np.all((e >= lo) & (e <= hi))
        s = np.exp2(e.astype(np.float64)).repeat(32, 1)
    exact = n / s
    lo, hi = e4m3_rounding_interval(q.numpy()[ok])
    slack = np.abs(exact) * 2 * DELTA + 2.0 ** -148 / s
    assert np.all((exact >= lo - slack) & (exact <= hi + slack))


# a step beyond 512 rows; one wave a row up to 2048 columns, four above; the last vectors of a thread partly empty
WIDTHS = {"bf16": (520, 2048, 2056, 8192, 8200, 16376), "int8": (640, 1992, 2176, 7168, 8320, 16384),
          "fp8": (640, 2048, 2176, 7168, 8320, 16384), "mxfp8": (544, 2016, 2080, 8192, 8224, 16352)}


@pytest.mark.parametrize("fmt,H", [(f, h) for f, hs in WIDTHS.items() for h in hs])
@pytest.mark.parametrize("residual,weight", [("none", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_many_rows(fmt, H, residual, weight):
    """Among them rows of zeros, with an infinity, a NaN, and squares that overflow fp32."""
    T = 513 if H > 2048 else 1031
    say("norm many rows", fmt, T, H, residual, weight)
    x, r, w = make(T, H, residual, weight, seed=H)
    x[3] = 0
    if r is not None:
        r[3] = 0
    x[4, H - 1], x[5, 0] = INF, NAN
    x[6] = (x[6].float() * 2.0 ** 100).bfloat16()
    x[7, H // 2] = 3e38
    x[T - 1, H - 1] = -3e38
    check(x, r, w, 1e-6, fmt, run(x, r, w, 1e-6, fmt))


@pytest.mark.parametrize("H", [2048, 7168, 16384])
def test_row_counts_that_pick_other_row_layouts(H):
    """Up to 512 rows and beyond, a row's squares are summed in another order: v is equal, n within twice DELTA."""
    T = 600
    x, r, w = (t.cuda() for t in make(T, H, "f32", "f32", seed=H + 1))
    many = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_INT8, residual=r, want_norm=True)
    few = fm.add_rmsnorm_quant(x[:512], w, 1e-6, fm.NORM_INT8, residual=r[:512], want_norm=True)
    torch.cuda.synchronize()
    assert torch.equal(few[3], many[3][:512])
    s, t = few[1].double(), many[1][:512].double()
    assert ((s - t).abs() <= t * (2 * DELTA + 2.0 ** -22)).all()
    assert ((few[0].int() - many[0][:512].int()).abs() <= 1).all()
    a, b = few[2].double(), many[2][:512].double()
    assert ((a - b).abs() <= b.abs() * (2.0 ** -7 + 4 * DELTA)).all()


def test_ties_of_int8_codes_go_to_even():
    """A row whose scale is 1 and whose values are whole numbers and halves, exactly: codes round halves to even."""
    # H = 64, v of 64 entries +-c with mean square c^2 and eps far below its step: n = w * sign, w free
    H = 64
    x = torch.ones(1, H).bfloat16()
    x[0, 1::2] = -1.0
    w = torch.zeros(H)
    w[:12] = torch.tensor([127.0, 127.0, 0.5, 0.5, 1.5, 1.5, 2.5, 2.5, 63.5, 63.5, 126.5, 126.5])
    q, s, n, _ = run(x, None, w, 2.0 ** -60, "int8")      # mean square 1 + 2^-60 is 1 in fp32
    assert s.item() == 1.0 and torch.equal(n[0].float(), (x[0].float() * w).bfloat16().float())
    assert q[0, :12].tolist() == [127, -127, 0, 0, 2, -2, 2, -2, 64, -64, 126, -126]
    v = torch.zeros(1, 16, dtype=torch.bfloat16)
    v[0, :9] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5, -62.5])
    q, s = fm.quant_rows_int8(v.cuda())
    assert s.item() == 1.0 and q[0, :9].tolist() == [127, 0, 2, 2, 0, -2, -2, 64, -62]


@pytest.mark.parametrize("T", [1, 600])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_small_values_beside_squares_that_overflow(T, fmt):
    """One value of 2^66 in a row of 16384, whose root mean square is 2^59: values of 2^-66 still have their bits."""
    H = 16384
    say("norm wide range", T, fmt)
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, H).bfloat16()
    x[:, 100] = 2.0 ** 66
    r = (1 + torch.rand(T, H, generator=g)) * 2.0 ** -66
    r[:, 100] = 0
    w = 1 + 0.3 * torch.rand(H, generator=g)
    check(x, r, w, 1e-6, fmt, run(x, r, w, 1e-6, fmt))


@pytest.mark.parametrize("H", [256, 16384])
def test_eps_beside_squares_that_overflow(H):
    """A mean square of about 2^128 / H, and an eps as large."""
    g = torch.Generator().manual_seed(H)
    x = torch.zeros(5, H).bfloat16()
    x[:, 7] = 1.5 * 2.0 ** 64
    r = torch.randn(5, H, generator=g) * 2.0 ** 50
    w = 1 + 0.3 * torch.randn(H, generator=g)
    for eps in (2.0 ** 128 / H, 2.0 ** 126, 1.0):
        for fmt in FORMATS:
            check(x, r, w, eps, fmt, run(x, r, w, eps, fmt))


def test_smallest_eps():
    """Squares that fp32 holds as subnormals, or not at all, beside the smallest eps."""
    x = (torch.randn(6, 512, generator=torch.Generator().manual_seed(1)) * 2.0 ** -64).bfloat16()
    x[3] = (x[3].float() * 2.0 ** -8).bfloat16()
    w = torch.ones(512)
    for fmt in FORMATS:
        check(x, None, w, 2.0 ** -126, fmt, run(x, None, w, 2.0 ** -126, fmt))
    with pytest.raises(fm.Fp8MoeError, match="eps"):
        run(x, None, w, 2.0 ** -127, "fp8")
