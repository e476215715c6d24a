"""The int8 layer and its stages on the GPU against the float64 oracle.

Tolerances.  The int32 sums are exact, and their conversion, the two scales and the products add at most four fp32
roundings, so h is within 4 * 2^-24 relative.  act follows through SwiGLU (silu' <= 1.1) with the error of its
evaluation, (2 |g| + 12) * 2^-24 relative, and is then the bf16 rounding of a value in that band (half a step, 2^-8).
Row codes are rounded from act / s within 2^-22 relative of the exact quotient.  Y is bf16 of a value within
6 * 2^-24.  The layer's output is held to the fused tolerance of the other formats.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle import int8 as O8
from tests.gpu_helpers import assert_rows_close_to_oracle, say

pytestmark = pytest.mark.gpu

TILES = (16, 32, 64, 288)


class Problem:
    def __init__(self, T, H, I, E, K, seed=0, skew=0.0, drop=0.0, low=-127):
        g = torch.Generator().manual_seed(seed)
        self.dims = (T, H, I, E, K)
        self.x = torch.randint(low, 128, (T, H), generator=g, dtype=torch.int8)
        self.xs = torch.rand(T, generator=g) * 0.02 + 0.005
        self.w13 = torch.randint(low, 128, (E, 2 * I, H), generator=g, dtype=torch.int8)
        self.w2 = torch.randint(low, 128, (E, H, I), generator=g, dtype=torch.int8)
        self.w13s = (torch.rand(E, 2 * I, generator=g) + 0.5) * 0.02 / H ** 0.5
        self.w2s = (torch.rand(E, H, generator=g) + 0.5) * 0.02 / I ** 0.5
        logits = torch.randn(T, E, generator=g) - skew * torch.log(torch.arange(1, E + 1.0))
        w, ids = torch.softmax(logits, 1).topk(K, dim=1)
        self.ids, self.tw = ids.int(), (w / w.sum(1, keepdim=True)).contiguous()
        if drop:
            self.ids[torch.rand(T, K, generator=g) < drop] = -1
        self.d = {k: getattr(self, k).cuda() for k in ("x", "xs", "w13", "w13s", "w2", "w2s", "ids", "tw")}
        self._packed = None

    def packed(self):
        if self._packed is None:
            self._packed = fm.pack_weights(self.d["w13"]), fm.pack_weights(self.d["w2"])
        return self._packed

    def run(self, tile_m=-1, packed=False, **kw):
        d = self.d
        w13, w2 = self.packed() if packed else (d["w13"], d["w2"])
        out = fm.moe_fused_int8(d["x"], d["xs"], w13, d["w13s"], w2, d["w2s"], d["ids"], d["tw"], tile_m=tile_m,
                                weight_layout=int(packed), **kw)
        torch.cuda.synchronize()
        return out

    def oracle(self):
        n = lambda t: t.numpy()
        return O8.moe_reference_int8(n(self.x), n(self.xs), n(self.w13), n(self.w13s), n(self.w2), n(self.w2s),
                                     n(self.ids), n(self.tw))


LAYERS = [dict(T=16, H=256, I=128, E=4, K=2), dict(T=1, H=128, I=128, E=1, K=1), dict(T=1, H=2048, I=768, E=16, K=8),
          dict(T=33, H=640, I=384, E=8, K=3, skew=1.2), dict(T=257, H=384, I=256, E=3, K=2, skew=1.2),
          dict(T=700, H=256, I=640, E=5, K=2, skew=1.2, drop=0.3), dict(T=65, H=896, I=128, E=300, K=2),
          dict(T=1300, H=512, I=256, E=2, K=1),
          # more experts than one round of the tile kernels' search, some of more than one tile
          dict(T=1700, H=128, I=128, E=600, K=2, skew=1.2), dict(T=2100, H=128, I=128, E=1024, K=1, skew=1.5),
          # a handful of rows: without routing, the largest of them, with dropped slots and beyond
          dict(T=1, H=384, I=1408, E=64, K=8), dict(T=2, H=512, I=768, E=128, K=8, skew=1.2),
          dict(T=5, H=128, I=2048, E=128, K=3, drop=0.4), dict(T=16, H=256, I=128, E=128, K=1),
          dict(T=17, H=256, I=4224, E=136, K=1), dict(T=1, H=256, I=128, E=128, K=9), dict(T=300, H=1152, I=896, E=1, K=1)]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_layer_matches_oracle_on_all_tiles_and_layouts(case):
    p = Problem(seed=3, **case)
    ref = p.oracle()
    first = None
    for packed in (False, True):
        for tm in (-1,) + TILES:
            say("int8 layer", case, "packed", packed, "tile_m", tm)
            out = p.run(tm, packed)
            if first is None:
                first = out
                assert_rows_close_to_oracle(out, ref, f"int8 {case}")
            assert torch.equal(out, first), f"packed={packed} tile_m={tm} differs"
    assert torch.equal(p.run(), first)


@pytest.mark.parametrize("align", [16, 64, 128])
@pytest.mark.parametrize("tile_m", TILES)
def test_stages(align, tile_m):
    p = Problem(90, 384, 256, 6, 2, seed=5, skew=0.8, drop=0.1, low=-128)
    T, H, I, E, K = p.dims
    d = p.d
    say("int8 stages", align, tile_m)
    r = fm.route_permute(d["ids"], E, align)
    act = fm.gemm1_swiglu_int8(d["x"], d["xs"], d["w13"], d["w13s"], r, T, K, align, tile_m=tile_m)
    q, qs = fm.quant_rows_int8(act, route=r)
    Y = fm.gemm2_weighted_int8(q, qs, d["w2"], d["w2s"], r, d["tw"], T, K, align, tile_m=tile_m)
    out = fm.combine(Y, d["ids"], E)
    torch.cuda.synchronize()
    fused = p.run().cpu().double().numpy()
    total, size = np.zeros((T, H)), np.zeros((T, H))
    src = r["sorted_src"].cpu().numpy()
    pos = np.flatnonzero(src >= 0)
    s = src[pos]
    e = p.ids.numpy().reshape(-1)[s]
    a = act.cpu().double().numpy()
    qn, qsn, Yn = q.cpu().double().numpy(), qs.cpu().double().numpy(), Y.cpu().double().numpy()
    for x in range(E):
        rows = pos[e == x]
        if not rows.size:
            continue
        tok = src[rows] // K
        h = O8.int8_product(p.x.numpy()[tok], p.xs.numpy()[tok], p.w13.numpy()[x], p.w13s.numpy()[x])
        want = O8.swiglu(h)
        g, u = np.abs(h[:, :I]), np.abs(h[:, I:])
        band = 4 * 2.0 ** -24 * (1.1 * g * u + np.abs(want)) + np.abs(want) * (2 * g + 12) * 2.0 ** -24
        assert np.all(np.abs(a[rows] - want) <= band + (np.abs(want) + band) * 2.0 ** -8)
        code, sc = O8.quantize_rows_int8(a[rows])
        assert np.all(np.abs(qsn[rows] - sc) <= sc * 2.0 ** -23)
        exact = a[rows] / qsn[rows][:, None]
        assert np.all(np.abs(qn[rows] - exact) <= 0.5 + np.abs(exact) * 2.0 ** -22)
        y = O8.int8_product(qn[rows], qsn[rows], p.w2.numpy()[x], p.w2s.numpy()[x])
        y *= p.tw.numpy().astype(np.float64).reshape(-1)[src[rows]][:, None]
        assert np.all(np.abs(Yn[src[rows]] - y) <= np.abs(y) * (2.0 ** -8 + 6 * 2.0 ** -24) + 1e-38)
        np.add.at(total, tok, y)
        np.add.at(size, tok, np.abs(y))
    # the layer keeps these few rows in fp32: its output is one bf16 rounding of their sum (K fp32 roundings of it)
    assert np.all(np.abs(fused - total) <= np.abs(total) * 2.0 ** -8 + size * (6 + K) * 2.0 ** -23)
    # the stages' Y is bf16: one rounding more per slot
    assert np.all(np.abs(out.cpu().double().numpy() - total) <= np.abs(total) * 2.0 ** -8 + size * 2.0 ** -8 * 1.01)
    # rows of padding and of dropped slots are left alone
    pad = np.flatnonzero(src < 0)
    assert not a[pad].any() and not qn[pad].any() and not qsn[pad].any()
    assert not Yn[p.ids.numpy().reshape(-1) < 0].any()


@pytest.mark.parametrize("T,H,I,E,K,skew,drop", [
    (400, 512, 256, 1, 1, 0.0, 0.0), (4096, 256, 640, 1, 1, 0.0, 0.0), (4100, 128, 1024, 1, 1, 0.0, 0.0),
    (4097, 256, 2048, 1, 1, 0.0, 0.1), (900, 256, 512, 3, 2, 1.2, 0.3), (300, 384, 1152, 20, 4, 1.2, 0.0),
    (597, 256, 1024, 34, 7, 1.2, 0.0), (129, 640, 384, 2, 1, 0.0, 0.0), (65, 128, 128, 9, 9, 0.0, 0.5)])
def test_few_tiles(T, H, I, E, K, skew, drop):
    """Launches whose tiles leave CUs without work: their heights and their order over the XCDs change no bit."""
    say("int8 few tiles", T, H, I, E, K, skew, drop)
    p = Problem(T, H, I, E, K, seed=T, skew=skew, drop=drop)
    ref = p.run(tile_m=32)
    for packed in (False, True):
        assert torch.equal(p.run(tile_m=288, packed=packed), ref)
        assert torch.equal(p.run(packed=packed), ref)
    if T * K < 1000:
        assert_rows_close_to_oracle(ref, p.oracle(), "int8 few tiles")


@pytest.mark.parametrize("H,low", [(16384, -128), (16256, -127)])
def test_largest_sums_are_exact(H, low):
    """Every product at its largest: the int32 sums reach 16384 * 128 * 128 = 2^28."""
    I = 128
    p = Problem(17, H, I, 2, 1, seed=1)
    p.d["x"].fill_(low)
    p.d["w13"].fill_(low)
    p.d["xs"].fill_(2.0 ** -14)
    p.d["w13s"].fill_(2.0 ** -14)
    r = fm.route_permute(p.d["ids"], 2, 16)
    act = fm.gemm1_swiglu_int8(p.d["x"], p.d["xs"], p.d["w13"], p.d["w13s"], r, 17, 1, 16)
    torch.cuda.synchronize()
    h = H * low * low * 2.0 ** -28
    want = h / (1 + np.exp(-h)) * h
    live = r["sorted_src"].cpu() >= 0
    assert np.all(np.abs(act.cpu()[live].double().numpy() - want) <= want * (2.0 ** -8 + 40 * 2.0 ** -24))


@pytest.mark.parametrize("T,E", [(4, 64), (90, 4)])
def test_repeated_and_foreign_experts(T, E):
    """The same expert in several slots of a token, and ids on both sides of [0, E)."""
    p = Problem(T, 256, 128, E, 4, seed=6)
    p.ids[:, 1] = p.ids[:, 0]
    p.ids[1] = 3
    p.ids[2, 2:] = torch.tensor([-7, E], dtype=torch.int32)
    p.d["ids"].copy_(p.ids)
    ref = p.oracle()
    first = p.run()
    assert_rows_close_to_oracle(first, ref, f"int8 repeated ids T={T}")
    for tm in TILES:
        assert torch.equal(p.run(tm, packed=True), first)


def test_all_slots_dropped_and_no_tokens():
    for E in (4, 256):      # routed, and a handful of rows
        p = Problem(8, 256, 128, E, 2)
        p.d["ids"].fill_(-1)
        for packed in (False, True):
            assert not p.run(packed=packed).any()
    d = p.d
    out = fm.moe_fused_int8(d["x"][:0], d["xs"][:0], d["w13"], d["w13s"], d["w2"], d["w2s"], d["ids"][:0],
                            d["tw"][:0])
    assert out.shape == (0, 256)


@pytest.mark.parametrize("T,E,tile_m", [(40, 4, 16), (40, 4, 64), (40, 4, 288), (13, 128, -1)])
def test_scales_without_numbers_stay_in_their_rows(T, E, tile_m):
    K = 2 if E == 4 else 1
    p = Problem(T, 256, 128, E, K, seed=2)
    clean = p.run(tile_m)
    p.d["xs"][7] = float("nan")
    p.d["xs"][11] = float("inf")
    out = p.run(tile_m)
    assert torch.isnan(out[[7, 11]]).all()
    keep = [t for t in range(T) if t not in (7, 11)]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("N", [8, 72, 256, 520, 1024, 1032, 2048, 4096, 4104, 16384])
def test_quant_rows(N):
    say("quant rows", N)
    g = torch.Generator().manual_seed(N)
    x = (torch.randn(37, N, generator=g) * torch.exp2(4 * torch.randn(37, 1, generator=g))).bfloat16()
    x[3] = 0
    x[4, N // 2] = float("nan")
    x[5, N - 1] = float("-inf")
    x[6] = (torch.randn(N, generator=g) * 2.0 ** -130).bfloat16()      # below the smallest scale
    x[7] = (torch.randn(N, generator=g).clamp(-4, 4) * 2.0 ** -112).bfloat16()
    q, s = fm.quant_rows_int8(x.cuda())
    torch.cuda.synchronize()
    q, s = q.cpu().double().numpy(), s.cpu().double().numpy()
    assert np.isnan(s[[4, 5]]).all() and not q[[4, 5]].any() and (s[[3, 6]] == 1).all() and not q[[3, 6]].any()
    ok = [r for r in range(37) if r not in (3, 4, 5, 6)]
    v = x[ok].double().numpy()
    _, want = O8.quantize_rows_int8(v)
    assert np.all(np.abs(s[ok] - want) <= want * 2.0 ** -23 + 2.0 ** -149)
    exact = v / s[ok][:, None]
    assert np.all(np.abs(q[ok] - exact) <= 0.5 + np.abs(exact) * 2.0 ** -22)


def test_more_rows_than_one_pass_of_the_grid():
    """Beyond 2^20 workgroups of 16 rows the quantiser strides."""
    rows = (1 << 24) + 5
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = (torch.arange(rows, device="cuda") % 128).bfloat16()
    q, s = fm.quant_rows_int8(x)
    torch.cuda.synchronize()
    want = torch.where(x[:, 3] > 0, 127, 0).to(torch.int8)
    assert torch.equal(q[:, 3], want) and not q[:, :3].any()


def test_streams_graph_and_poisoned_workspace():
    p = Problem(48, 512, 256, 8, 2, seed=9, skew=1.0)
    want = p.run(packed=True)
    T, H, I, E, K = p.dims
    ws = fm.alloc_workspace_int8(T, H, I, E, K, "cuda")
    for byte in (0, 0x7F, 0xFF):
        ws.fill_(byte)
        assert torch.equal(p.run(packed=True, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.run(packed=True)
    assert torch.equal(got, want)
    d = p.d
    w13, w2 = p.packed()
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(g):
        fm.moe_fused_int8(d["x"], d["xs"], w13, d["w13s"], w2, d["w2s"], d["ids"], d["tw"], out=out, workspace=ws,
                          weight_layout=1)
    for seed in (1, 2, 3):
        n = Problem(48, 512, 256, 8, 2, seed=seed)
        for k in ("x", "xs", "ids", "tw"):
            d[k].copy_(n.d[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, p.run(packed=True))


@pytest.mark.parametrize("T", [1024, 1025])
def test_rows_kept_in_fp32_and_in_bf16(T):
    """T * K * H at the border between the two: the same output to a bf16 step of each slot."""
    p = Problem(T, 1024, 128, 16, 4, seed=4)
    ref = p.oracle()
    first = p.run()
    assert_rows_close_to_oracle(first, ref, f"int8 Y T={T}")
    for tm in TILES:
        assert torch.equal(p.run(tm), first)


def test_offsets_beyond_32_bits():
    """Expert weights, and an expert's byte offset, beyond 2^32."""
    E, H, I = 40, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device="cuda", dtype=torch.int8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-127, 128, (3, H), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.full((3,), 0.01, device="cuda")
    w13s = torch.full((E, 2 * I), 1e-4, device="cuda")
    w2s = torch.full((E, H), 1e-4, device="cuda")
    ids = torch.tensor([[39, 0], [17, 39], [38, 37]], dtype=torch.int32, device="cuda")
    tw = torch.full((3, 2), 0.5, device="cuda")
    out = fm.moe_fused_int8(x, xs, w13, w13s, w2, w2s, ids, tw)
    torch.cuda.synchronize()
    ref = np.zeros((3, H))
    n = lambda t: t.cpu().numpy()
    for t in range(3):
        for e in ids[t].tolist():
            ref[t] += O8.moe_reference_int8(n(x[t:t + 1]), n(xs[t:t + 1]), n(w13[e:e + 1]), n(w13s[e:e + 1]),
                                            n(w2[e:e + 1]), n(w2s[e:e + 1]), np.zeros((1, 1), np.int32),
                                            np.full((1, 1), 0.5))[0]
    assert_rows_close_to_oracle(out, ref, "int8 far experts")


def test_refusals():
    p = Problem(8, 256, 128, 4, 2)
    d = p.d
    f = lambda **kw: fm.moe_fused_int8(**{**dict(x=d["x"], x_scale=d["xs"], w13=d["w13"], w13_scale=d["w13s"],
                                                 w2=d["w2"], w2_scale=d["w2s"], topk_ids=d["ids"],
                                                 topk_weights=d["tw"]), **kw})
    with pytest.raises(TypeError):
        f(x=d["x"].view(torch.uint8))
    with pytest.raises(TypeError):
        f(topk_ids=d["ids"].long())
    with pytest.raises(ValueError):
        f(x_scale=d["xs"][:7])
    with pytest.raises(ValueError):
        f(w13_scale=d["w13s"][:, :128].contiguous())
    with pytest.raises(ValueError):
        f(w2=d["w2"][:3])
    with pytest.raises(ValueError):
        f(x=d["x"].t().contiguous().t())
    with pytest.raises(ValueError):
        f(w2_scale=d["w2s"].cpu())
    with pytest.raises(ValueError):
        f(out=torch.empty(8, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fm.Fp8MoeError, match="workspace"):
        f(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for tm in (0, 8, 48, 512):
        with pytest.raises(fm.Fp8MoeError, match="tile_m"):
            f(tile_m=tm)
    flat = torch.zeros(8 * 256 + 16, dtype=torch.int8, device="cuda")
    with pytest.raises(fm.Fp8MoeError, match="aligned"):
        f(x=flat[1:1 + 8 * 256].view(8, 256))
    r = fm.route_permute(d["ids"], 4, 16)      # a routing of 4 experts is no routing of 3
    with pytest.raises(ValueError, match="padded_indptr"):
        fm.gemm1_swiglu_int8(d["x"], d["xs"], d["w13"][:3], d["w13s"][:3], r, 8, 2, 16)
    act = fm.gemm1_swiglu_int8(d["x"], d["xs"], d["w13"], d["w13s"], r, 8, 2, 16)
    q, qs = fm.quant_rows_int8(act, route=r)
    with pytest.raises(ValueError, match="padded_indptr"):
        fm.gemm2_weighted_int8(q, qs, d["w2"][:3], d["w2s"][:3], r, d["tw"], 8, 2, 16)
    with pytest.raises(ValueError, match="rows"):
        fm.quant_rows_int8(act[:-1], route=r)
