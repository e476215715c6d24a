"""add_rmsnorm_quant on the GPU against the float64 oracle.

Tolerances.  v is exact: the stored stream must equal the oracle's bit for bit.  The kernel sums at most 64 squares
in one thread and joins at most 16 partial sums' worth of roundings, all of positive terms, so the mean square is
within 80 * 2^-24 relative; halved by the root, plus the roundings of the mean, eps, root, reciprocal and the two
products: n is within DELTA = 48 * 2^-24 relative.  bf16(n) adds half a step, 2^-8 relative.  Codes are held to the
rounding interval of n / scale for the scale the GPU stored.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle.norm import add_rmsnorm_reference
from tests.gpu_helpers import e4m3_rounding_interval, e8m0_exponent_range, say

pytestmark = pytest.mark.gpu

DELTA = 48 * 2.0 ** -24
FORMATS = {"bf16": fm.NORM_BF16, "fp8": fm.NORM_FP8, "mxfp8": fm.NORM_MXFP8, "int8": fm.NORM_INT8}


def make(T, H, residual="bf16", weight="bf16", seed=0, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    x = (x * torch.exp2(spread * torch.randn(T, H, generator=g))).bfloat16()
    r = None
    if residual != "none":
        r = torch.randn(T, H, generator=g) * 3
        r = r.bfloat16() if residual == "bf16" else r
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x, r, (w.bfloat16() if weight == "bf16" else w)


def run(x, r, w, eps, fmt, **kw):
    c = lambda t: None if t is None else t.cuda()
    out = fm.add_rmsnorm_quant(c(x), c(w), eps, FORMATS[fmt], residual=c(r), **kw)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in out]


def f64(t):
    return t.double().numpy()


def check(x, r, w, eps, fmt, q, scale, norm, v):
    T, H = x.shape
    vr, n = add_rmsnorm_reference(f64(x), None if r is None else f64(r), f64(w), eps, r is not None and
                                  r.dtype == torch.bfloat16)
    if r is None:
        assert v is None
    else:
        assert np.array_equal(f64(v), vr)
    if norm is not None:
        assert np.all(np.abs(f64(norm) - n) <= np.abs(n) * (2.0 ** -8 + 2 * DELTA) + 1e-38)
    if fmt == "fp8":
        s = f64(scale).repeat(128, 1)
        amax = np.abs(n).reshape(T, -1, 128).max(2)
        want = np.where(amax > 0, amax / 448, 1.0)
        assert np.all(np.abs(f64(scale) - want) <= want * (DELTA + 2.0 ** -23))
    elif fmt == "mxfp8":
        amax = np.abs(n).reshape(T, -1, 32).max(2)
        lo, hi = e8m0_exponent_range(amax * (1 - DELTA), amax * (1 + DELTA))
        e = scale.numpy().astype(np.int64) - 127
        assert np.all((e >= lo) & (e <= hi))
        s = np.exp2(e.astype(np.float64)).repeat(32, 1)
    elif fmt == "int8":
        amax = np.abs(n).max(1)
        want = np.where(amax > 0, amax / 127, 1.0)
        assert np.all(np.abs(f64(scale) - want) <= want * (DELTA + 2.0 ** -23))
        exact = n / f64(scale)[:, None]
        assert np.all(np.abs(f64(q) - exact) <= 0.5 + np.abs(exact) * 2 * DELTA)
        return
    else:
        assert q is None and scale is None
        return
    exact = n / s
    lo, hi = e4m3_rounding_interval(q.numpy())
    slack = np.abs(exact) * 2 * DELTA + 2.0 ** -148 / s      # and the step of fp32's subnormals
    assert np.all((exact >= lo - slack) & (exact <= hi + slack))


SHAPES = [(1, 128), (1, 7168), (3, 512), (5, 640), (2, 2048), (7, 2176), (33, 7168), (2, 8192), (3, 8320),
          (1, 16384), (1030, 256)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("T,H", SHAPES)
def test_shapes(T, H, fmt):
    say("norm", fmt, T, H)
    x, r, w = make(T, H, seed=H + T)
    check(x, r, w, 1e-6, fmt, *run(x, r, w, 1e-6, fmt, want_norm=True))


@pytest.mark.parametrize("fmt,H", [("bf16", 8), ("int8", 8), ("int8", 72), ("bf16", 4104), ("mxfp8", 32),
                                   ("mxfp8", 96), ("mxfp8", 2080), ("int8", 16376)])
def test_odd_widths(fmt, H):
    say("norm width", fmt, H)
    x, r, w = make(9, H, residual="f32", weight="f32", seed=H)
    check(x, r, w, 1e-5, fmt, *run(x, r, w, 1e-5, fmt, want_norm=True))


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("residual", ["none", "bf16", "f32"])
@pytest.mark.parametrize("weight", ["bf16", "f32"])
def test_types(fmt, residual, weight):
    say("norm types", fmt, residual, weight)
    x, r, w = make(17, 1280, residual, weight, seed=4, spread=2.0)
    out = run(x, r, w, 1e-6, fmt)
    assert (out[2] is None) == (fmt != "bf16")
    check(x, r, w, 1e-6, fmt, *out)


def test_int8_ties_round_to_even():
    """n = v exactly (weight = rms): codes of v / s with s = 1 are v rounded to even."""
    v = torch.zeros(1, 64)
    v[0, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5])
    x = v.bfloat16()
    rms = float(torch.sqrt((v.double() ** 2).mean() + 1e-6))
    w = torch.full((64,), rms)
    q, s, _, _ = run(x, None, w, 1e-6, "int8")
    exact = v[0].double().numpy() / float(s[0]) * 1.0
    assert np.all(np.abs(q[0].numpy() - exact) <= 0.5 + np.abs(exact) * 4 * DELTA)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_zero_rows_and_zero_blocks(fmt):
    say("norm zeros", fmt)
    x, r, w = make(4, 256, residual="none", seed=9)
    x[1] = 0
    x[2, 128:] = 0
    q, scale, norm, _ = run(x, r, w, 1e-6, fmt, want_norm=True)
    check(x, r, w, 1e-6, fmt, q, scale, norm, None)
    assert torch.all(norm[1] == 0)
    if fmt == "fp8":
        assert torch.all(scale[1] == 1) and scale[2, 1] == 1
    if fmt == "mxfp8":
        assert torch.all(scale[1] == 0)
    if fmt == "int8":
        assert scale[1] == 1 and torch.all(q[1] == 0)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("H", [256, 2560])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_rows_without_numbers(fmt, H, bad):
    say("norm bad", fmt, H, bad)
    x, r, w = make(5, H, residual="bf16", seed=3)
    clean = run(x, r, w, 1e-6, fmt, want_norm=True)
    x[2, 77] = bad
    q, scale, norm, v = run(x, r, w, 1e-6, fmt, want_norm=True)
    assert torch.isnan(norm[2]).all()
    if fmt == "fp8":
        assert torch.isnan(scale[2]).all() and torch.all(q[2] == 0x7F)
    elif fmt == "mxfp8":
        assert torch.all(scale[2] == 255) and torch.all(q[2] == 0x7F)
    elif fmt == "int8":
        assert torch.isnan(scale[2]) and torch.all(q[2] == 0)
    keep = [0, 1, 3, 4]
    for a, b in zip((q, scale, norm, v), clean):   # the other rows do not change
        if a is not None:
            assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "int8"])
def test_weight_without_numbers(fmt):
    x, r, w = make(3, 384, residual="none", weight="f32", seed=8)
    w[130] = float("nan")
    q, scale, norm, _ = run(x, r, w, 1e-6, fmt, want_norm=True)
    assert torch.isnan(norm[:, 130]).all() and torch.isfinite(norm[:, 131:].float()).all()
    if fmt == "int8":
        assert torch.isnan(scale).all() and torch.all(q == 0)
    elif fmt == "fp8":
        assert torch.isnan(scale[:, 1]).all() and torch.isfinite(scale[:, [0, 2]]).all()
    else:
        assert torch.all(scale[:, 4] == 255) and torch.all(scale[:, [0, 1, 2, 3, 5, 6]] != 255)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_squares_beyond_fp32(fmt):
    """|v| up to 3e38: the squares overflow fp32, the norm does not."""
    say("norm large", fmt)
    x, r, w = make(3, 640, residual="f32", weight="f32", seed=12)
    x[0] = (x[0].float() * 2.0 ** 120).bfloat16()
    x[1, 5] = 3e38
    r[0] *= 2.0 ** 100
    check(x, r, w, 1e-6, fmt, *run(x, r, w, 1e-6, fmt, want_norm=True))


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_in_place_residual_and_given_outputs(fmt):
    x, r, w = (t.cuda() for t in make(6, 1024, residual="f32", seed=2))
    q, s, n, v = fm.add_rmsnorm_quant(x, w, 1e-6, FORMATS[fmt], residual=r, want_norm=True)
    r2 = r.clone()
    kw = {} if fmt == "bf16" else {"q": torch.empty_like(q), "scale": torch.empty_like(s)}
    out = fm.add_rmsnorm_quant(x, w, 1e-6, FORMATS[fmt], residual=r2, residual_out=r2, norm_out=torch.empty_like(n),
                               **kw)
    assert out[3] is r2
    for a, b in zip(out, (q, s, n, v)):
        if b is not None:
            assert torch.equal(a, b)


def test_rows_do_not_depend_on_their_neighbours():
    """Row counts that pick other row layouts give the same bits."""
    x, r, w = (t.cuda() for t in make(4097, 512, seed=6))
    big = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_FP8, residual=r, want_norm=True)
    for t0, t1 in ((0, 1), (5, 8), (100, 229), (4096, 4097)):
        part = fm.add_rmsnorm_quant(x[t0:t1], w, 1e-6, fm.NORM_FP8, residual=r[t0:t1], want_norm=True)
        for a, b in zip(part, big):
            assert torch.equal(a, b[t0:t1])


def test_stream_and_graph():
    """On a side stream, and captured and replayed with new inputs."""
    x, r, w = (t.cuda() for t in make(40, 2048, seed=1))
    want = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_INT8, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_INT8, residual=r)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_INT8, residual=r)
    for seed in (5, 6, 7):
        x2, r2, _ = make(40, 2048, seed=seed)
        x.copy_(x2)
        r.copy_(r2)
        g.replay()
        torch.cuda.synchronize()
        want = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_INT8, residual=r)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(out[3], want[3])


def test_refusals():
    x, r, w = (t.cuda() for t in make(4, 256))
    f = fm.add_rmsnorm_quant
    with pytest.raises(TypeError):
        f(x.float(), w, 1e-6, fm.NORM_FP8)
    with pytest.raises(TypeError):
        f(x, w.half(), 1e-6, fm.NORM_FP8)
    with pytest.raises(ValueError):
        f(x, w[:-8], 1e-6, fm.NORM_FP8)
    with pytest.raises(ValueError):
        f(x.t(), w, 1e-6, fm.NORM_FP8)
    with pytest.raises(ValueError):
        f(x, w, 1e-6, fm.NORM_FP8, residual=r[:3])
    with pytest.raises(ValueError):
        f(x, w, 1e-6, fm.NORM_FP8, residual_out=r)
    with pytest.raises(ValueError):
        f(x, w, 1e-6, fm.NORM_BF16, q=torch.empty(4, 256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        f(x, w.cpu(), 1e-6, fm.NORM_FP8)
    flat = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fm.Fp8MoeError, match="aligned"):
        f(flat[1:1 + 4 * 256].view(4, 256), w, 1e-6, fm.NORM_FP8)
    with pytest.raises(fm.Fp8MoeError, match="overlap"):
        f(x, w, 1e-6, fm.NORM_BF16, norm_out=x)
    with pytest.raises(fm.Fp8MoeError, match="eps"):
        f(x, w, 0.0, fm.NORM_FP8)
    empty = f(x[:0], w, 1e-6, fm.NORM_FP8, residual=r[:0])
    assert empty[0].shape == (0, 256) and empty[3].shape == (0, 256)
