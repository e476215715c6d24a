"""The products and the block quantiser as they are used: in a row, in captured graphs, on other streams and threads,
with offsets beyond 32 bits, at the largest sizes, and with every tile height.

Whole-number operands and power-of-two scales make every sum exact (see test_gpu_products), so outputs are compared
for equality, with the same product in float64 on the GPU where it is large.  The layer's comparisons use the
fused-layer tolerance: the same operands in the same formats.
"""

import threading

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
import synth
from oracle.moe import moe_reference
from tests.gpu_helpers import assert_rows_close_to_oracle, say

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def nb(n):
    return -(-n // 128)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(g, *shape, dtype=E4M3, top=2):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(torch.float16).to(dtype)


def powers(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def product64(a, sa, b, sb):
    """The product in float64, block by block of K."""
    y = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    if sa is None:
        return a.double() @ b.double().t()
    row = torch.arange(b.shape[0], device=a.device) // 128
    for k in range(nb(a.shape[1])):
        c = slice(128 * k, 128 * k + 128)
        y += (a[:, c].double() * sa[:, k].double()[:, None]) @ (b[:, c].double() * sb[row, k].double()[:, None]).t()
    return y


def gemm_operands(g, M, N, K):
    return whole(g, M, K), powers(g, M, nb(K)), whole(g, N, K), powers(g, nb(N), nb(K))


# ---------------------------------------------------------------- in a row

def test_experts_over_ragged_rows_match_the_layer():
    """Rows sorted by expert without padding -> gate and up -> SwiGLU and quantisation -> down -> weighted sum: what
    the fused layer computes."""
    d = synth.TINY
    p = synth.moe_problem(70, d["H"], d["I"], d["E"], d["K"], synth.CFG_TINY)
    pd = p.to("cuda")
    K = d["K"]
    say("experts over ragged rows")
    route = fm.route_permute(pd.topk_ids, d["E"], 16)
    flat = pd.topk_ids.view(-1)
    order = torch.sort(flat, stable=True).indices            # every slot is valid here
    token = order // K
    w13, w2 = fm.pack_weights(pd.w13_q), fm.pack_weights(pd.w2_q)
    for tiled in (False, True):
        layout = fm.WEIGHTS_MFMA_TILED if tiled else fm.WEIGHTS_ROW_MAJOR
        h = fm.grouped_gemm_fp8_ragged(pd.x_q[token].contiguous(), pd.x_s[token].contiguous(),
                                       w13 if tiled else pd.w13_q, pd.w13_s, route["m_indptr"],
                                       out_dtype=torch.float32, weight_layout=layout)
        q, s = fm.quant_fp8_blocks(h, gated=True)
        y = fm.grouped_gemm_fp8_ragged(q, s, w2 if tiled else pd.w2_q, pd.w2_s, route["m_indptr"],
                                       out_dtype=torch.float32, weight_layout=layout)
        out = torch.zeros(p.x_q.shape[0], d["H"], device="cuda")
        out.index_add_(0, token, y * pd.topk_weights.view(-1)[order][:, None])
        _, ref = moe_reference(p.x_q.numpy(), p.x_s.numpy(), p.w13_q.numpy(), p.w13_s.numpy(), p.w2_q.numpy(),
                               p.w2_s.numpy(), p.topk_ids.numpy(), p.topk_weights.numpy())
        assert_rows_close_to_oracle(out.bfloat16(), ref, "ragged experts")


@pytest.mark.parametrize("T", [1, 37, 300])
def test_shared_expert_onto_the_routed_ones(T):
    """Norm -> dense gate and up -> SwiGLU and quantisation -> dense down, added to what the layer gave; the dense part
    alone equals the layer with one expert of weight 1."""
    H, I = 512, 384
    g = gen(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    q, s, _, _ = fm.add_rmsnorm_quant(x, w, 1e-6, fm.NORM_FP8)
    w13 = (torch.randn(2 * I, H, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4M3)
    w2 = (torch.randn(H, I, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4M3)
    s13 = torch.rand(2 * I // 128, H // 128, generator=g, device="cuda") * 5e-4
    s2 = torch.rand(H // 128, I // 128, generator=g, device="cuda") * 5e-4
    routed = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    say("shared expert", T)
    h = fm.gemm_fp8_blocks(q, s, w13, s13, out_dtype=torch.float32)
    hq, hs = fm.quant_fp8_blocks(h, gated=True)
    alone = fm.gemm_fp8_blocks(hq, hs, w2, s2)
    out = fm.gemm_fp8_blocks(hq, hs, w2, s2, addend=routed, out=routed.clone())
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    layer = fm.moe_fused_fp8(q, s, w13[None].view(torch.uint8), s13[None], w2[None].view(torch.uint8), s2[None], ids,
                             torch.ones(T, 1, device="cuda"))
    torch.cuda.synchronize()
    # both sides are within the fused-layer tolerance of the exact layer: codes of the intermediate may fall
    # to either side of a tie, and both round once to bf16
    rel = ((alone.double() - layer.double()).norm() / layer.double().norm()).item()
    assert rel <= 1e-2, rel
    want = product64(hq.view(E4M3), hs, w2, s2)
    err = (out.double() - (want + routed.double())).abs()
    assert torch.all(err <= (want.abs() + routed.double().abs()) * 2.0 ** -8 + 2.0 ** -13 * product64(
        hq.view(E4M3).float().abs().to(E4M3), hs, w2.float().abs().to(E4M3), s2))


# ---------------------------------------------------------------- graphs, streams, threads

CALLS = {
    "gemm": lambda s: fm.gemm_fp8_blocks(*s["dense"], out=s["o1"], workspace=s["ws"]),
    "gemm parts": lambda s: fm.gemm_fp8_blocks(*s["deep"], out=s["o2"], workspace=s["ws"]),
    "gemm parts of tiles": lambda s: fm.gemm_fp8_blocks(*s["wide"], out=s["o5"], workspace=s["ws"]),
    "ragged": lambda s: fm.grouped_gemm_fp8_ragged(*s["grouped"], s["ptr"], out=s["o3"]),
    "ragged bf16": lambda s: fm.grouped_gemm_bf16_ragged(*s["bf16"], s["ptr"], out=s["o4"]),
    "quant": lambda s: fm.quant_fp8_blocks(s["x"], gated=True, q=s["q"], scale=s["qs"]),
}


def state(seed):
    g = gen(seed)
    s = {"dense": gemm_operands(g, 700, 520, 1040), "deep": gemm_operands(g, 20, 300, 7168),
         "wide": gemm_operands(g, 300, 500, 7168)}
    a, sa, _, _ = gemm_operands(g, 500, 128, 400)
    s["grouped"] = a, sa, whole(g, 3, 200, 400), powers(g, 3, 2, 4)
    s["bf16"] = whole(g, 500, 400, dtype=torch.bfloat16), whole(g, 3, 200, 400, dtype=torch.bfloat16)
    s["ptr"] = torch.tensor([0, 100, 100, 490], dtype=torch.int32, device="cuda")
    s["x"] = torch.randn(300, 512, generator=g, device="cuda").bfloat16()
    z = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device="cuda")
    s["o1"], s["o2"], s["o3"], s["o4"], s["o5"] = z(700, 520), z(20, 300), z(500, 200), z(500, 200), z(300, 500)
    s["q"] = torch.zeros(300, 256, dtype=torch.uint8, device="cuda")
    s["qs"] = torch.zeros(300, 2, device="cuda")
    s["ws"] = torch.zeros(max(fm.gemm_workspace_size(700, 520, 1040), fm.gemm_workspace_size(20, 300, 7168),
                              fm.gemm_workspace_size(300, 500, 7168), 1), dtype=torch.uint8, device="cuda")
    return s


def outputs(s):
    return [s[k].clone() for k in ("o1", "o2", "o3", "o4", "o5", "q", "qs")]


def clear(s):
    for k in ("o1", "o2", "o3", "o4", "o5", "q", "qs"):
        s[k].zero_()


def run_all(s):
    for f in CALLS.values():
        f(s)


def expected(s):
    run_all(s)
    torch.cuda.synchronize()
    want = outputs(s)
    for k, ops in (("o1", "dense"), ("o2", "deep"), ("o5", "wide")):
        assert torch.equal(s[k], product64(*s[ops]).to(torch.bfloat16)), ops
    return want


def test_captured_calls_replay():
    s = state(1)
    say("graph")
    want = expected(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(s)
    for i in range(4):
        clear(s)
        if i % 2:
            s["ws"].fill_(255)                      # nothing of it is read before it is written
            fm.gemm_fp8_blocks(*s["deep"])           # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(s), want)), i


def test_two_captured_graphs_share_a_workspace():
    s, t = state(2), state(3)
    t["ws"] = s["ws"]
    ws, wt = expected(s), expected(t)
    graphs = []
    for u in (s, t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_all(u)
        graphs.append(graph)
    for _ in range(3):
        clear(s)
        clear(t)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(s), ws))
        assert all(torch.equal(a, b) for a, b in zip(outputs(t), wt))


def test_side_streams_and_threads():
    states = [state(4 + i) for i in range(3)]
    want = [expected(s) for s in states]
    for s in states:
        clear(s)
    torch.cuda.synchronize()
    errors = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    run_all(s)
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    say("threads")
    threads = [threading.Thread(target=work, args=(s,)) for s in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for s, w in zip(states, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs(s), w))


# ---------------------------------------------------------------- tile heights and kernels

@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("lo,hi,N,K", [(97, 256, 1536, 1024), (1, 130, 1000, 400), (1, 70, 1200, 640), (1, 9, 300, 272)])
def test_ragged_every_height(fmt, tiled, lo, hi, N, K):
    """Groups of every size between lo and hi: every number of sub-tiles of the tile kernels."""
    E = 128
    g = gen(lo + hi)
    if tiled:
        N, K = -(-N // 16) * 16, -(-K // 128) * 128
    sizes = torch.randint(lo, hi + 1, (E,), generator=g, device="cuda")
    sizes[:min(E, hi - lo + 1)] = torch.arange(lo, min(hi, lo + E - 1) + 1, device="cuda")
    ptr = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), sizes.cumsum(0)]).to(torch.int32)
    ends = ptr.tolist()
    t = E4M3 if fmt == "fp8" else torch.bfloat16
    a, b = whole(g, ends[-1], K, dtype=t), whole(g, E, N, K, dtype=t)
    w = fm.pack_weights(b).view(t) if tiled else b
    layout = fm.WEIGHTS_MFMA_TILED if tiled else fm.WEIGHTS_ROW_MAJOR
    say("every height", fmt, tiled, lo, hi, N, K)
    sa = sb = None
    if fmt == "fp8":
        sa, sb = powers(g, ends[-1], nb(K)), powers(g, E, nb(N), nb(K))
        out = fm.grouped_gemm_fp8_ragged(a, sa, w, sb, ptr, out_dtype=torch.float32, weight_layout=layout)
    else:
        out = fm.grouped_gemm_bf16_ragged(a, w, ptr, out_dtype=torch.float32, weight_layout=layout)
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        want = product64(a[r], None if sa is None else sa[r], b[e], None if sb is None else sb[e])
        assert torch.equal(out[r].double(), want), f"group {e} of {ends[e + 1] - ends[e]} rows"


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("sizes,N,K", [([9000, 3, 0, 7100, 300, 40, 3557], 1500, 528), ([20000], 1536, 512),
                                       ([30, 60, 0, 90] * 75 + [22000, 2049], 1536, 512),
                                       ([2304] * 8 + [1, 2305, 100], 2048, 384)])
def test_ragged_high_and_low_groups(fmt, sizes, N, K):
    """Groups of more than eight tiles beside low ones, whose tiles are dealt out: every row, and none behind."""
    E, rows = len(sizes), sum(sizes)
    g = gen(E + rows)
    ptr = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    t = E4M3 if fmt == "fp8" else torch.bfloat16
    a, b = whole(g, rows + 5, K, dtype=t), whole(g, E, N, K, dtype=t)
    out = torch.full((rows + 5, N), 7.5, dtype=torch.float32, device="cuda")
    say("high and low groups", fmt, E, rows)
    sa = sb = None
    if fmt == "fp8":
        sa, sb = powers(g, rows + 5, nb(K)), powers(g, E, nb(N), nb(K))
        fm.grouped_gemm_fp8_ragged(a, sa, b, sb, ptr, out=out)
    else:
        fm.grouped_gemm_bf16_ragged(a, b, ptr, out=out)
    ends = ptr.tolist()
    assert torch.all(out[rows:] == 7.5)
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        want = product64(a[r], None if sa is None else sa[r], b[e], None if sb is None else sb[e])
        assert torch.equal(out[r].double(), want), f"group {e} of {sizes[e]} rows"


@pytest.mark.parametrize("M,N,K", [(4096, 2000, 2048), (2500, 4100, 1040), (2048, 4096, 1936), (1111, 3900, 2064),
                                   (1111, 2000, 1936), (700, 516, 16384), (4100, 520, 4240),
                                   (512, 1500, 7168), (300, 500, 7184), (130, 260, 16384), (64, 500, 7168),
                                   (48, 4096, 2000), (30, 130, 4096), (20, 7170, 2064), (60, 7168, 2048), (5, 7168, 2048),
                                   (1, 33, 16384)])
@pytest.mark.parametrize("addend", [False, True])
def test_gemm_every_kernel(M, N, K, addend):
    """Sizes at which the cost model takes each of the kernels, in one part of K and in several."""
    g = gen(M + N)
    ops = gemm_operands(g, M, N, K)
    add = whole(g, M, N, dtype=torch.bfloat16) if addend else None
    say("every kernel", M, N, K, addend)
    want = product64(*ops)
    if addend:
        want += add.double()
    assert torch.equal(fm.gemm_fp8_blocks(*ops, addend=add, out_dtype=torch.float32).double(), want)
    assert torch.equal(fm.gemm_fp8_blocks(*ops, addend=add), want.to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(4096, 2000, 2048), (2500, 4112, 1152), (8200, 4096, 2048), (1111, 2000, 1920),
                                   (300, 7168, 2048), (700, 528, 8192), (300, 512, 7168), (130, 272, 16384),
                                   (33, 4096, 2048)])
def test_gemm_every_kernel_tiled(M, N, K):
    g = gen(M + K)
    a, sa, b, sb = gemm_operands(g, M, N, K)
    say("every kernel tiled", M, N, K)
    out = fm.gemm_fp8_blocks(a, sa, fm.pack_weights(b[None]).view(E4M3)[0], sb, out_dtype=torch.float32,
                             weight_layout=fm.WEIGHTS_MFMA_TILED)
    assert torch.equal(out.double(), product64(a, sa, b, sb))


@pytest.mark.parametrize("M,N,K", [(3, 70, 65536), (100, 300, 65536), (3, 65536, 128), (200, 65536, 48), (1, 65536, 2048)])
def test_gemm_largest_sides(M, N, K):
    g = gen(K + N)
    ops = gemm_operands(g, M, N, K)
    say("largest sides", M, N, K)
    assert torch.equal(fm.gemm_fp8_blocks(*ops, out_dtype=torch.float32).double(), product64(*ops))


# ---------------------------------------------------------------- offsets beyond 32 bits

def test_gemm_far_rows():
    """a of 4.5 GiB and out of 4.3 GiB: the last rows and some around 2^32 against the same rows alone."""
    M, N, K = 2_200_000, 1024, 2176
    g = gen(1)
    a = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    for r in range(0, M, 200_000):
        a[r:r + 200_000] = whole(g, 200_000, K).view(torch.uint8)
    sa, b, sb = powers(g, M, nb(K)), whole(g, N, K), powers(g, nb(N), nb(K))
    say("far rows")
    out = fm.gemm_fp8_blocks(a, sa, b, sb)
    torch.cuda.synchronize()
    for r in (0, 2 ** 32 // K - 3, 2 ** 31 // N - 5, 2 ** 32 // (2 * N) - 3, M - 7):
        rows = slice(r, min(r + 7, M))
        assert torch.equal(out[rows], product64(a[rows].view(E4M3), sa[rows], b, sb).to(torch.bfloat16)), r


def test_ragged_far_groups():
    """Weights of 5 GiB: the last group's rows, tiles and streaming."""
    E, N, K = 640, 4096, 2048
    g = gen(2)
    b = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    b[0], b[-1] = whole(g, N, K).view(torch.uint8), whole(g, N, K).view(torch.uint8)
    sb = powers(g, E, nb(N), nb(K))
    for rows in (3, 300, 80_000):
        a, sa = whole(g, rows, K), powers(g, rows, nb(K))
        ptr = torch.full((E + 1,), 1, dtype=torch.int32, device="cuda")
        ptr[0], ptr[-1] = 0, rows
        say("far groups", rows)
        out = fm.grouped_gemm_fp8_ragged(a, sa, b, sb, ptr, out_dtype=torch.float32)
        assert torch.equal(out[:1].double(), product64(a[:1], sa[:1], b[0].view(E4M3), sb[0]))
        for r in (1, rows - 2):
            s = slice(max(r, 1), r + 2)
            assert torch.equal(out[s].double(), product64(a[s], sa[s], b[-1].view(E4M3), sb[-1])), (rows, r)


@pytest.mark.parametrize("rows", [1, 50, 4000, 2 ** 29 - 2 ** 21])
def test_ragged_overlapping_groups(rows):
    """512 groups of every row: more tiles than distinct groups could have, and with the most rows more than 2^31.
    What is written is a group's result (the groups are equal here), nothing behind the rows is."""
    E, N, K, mark = 1024, 16, 16, 99.0
    g = gen(rows)
    few = min(rows, 4096)
    a, sa = whole(g, few, K).repeat(rows // few, 1), powers(g, few, 1).repeat(rows // few, 1)
    b, sb = whole(g, 1, N, K).expand(E, N, K).contiguous(), powers(g, 1, 1, 1).expand(E, 1, 1).contiguous()
    ptr = torch.tensor([0, rows] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    out = torch.full((rows + 64, N), mark, dtype=torch.bfloat16, device="cuda")
    say("overlapping groups", rows)
    fm.grouped_gemm_fp8_ragged(a, sa, b, sb, ptr, out=out[:rows])
    torch.cuda.synchronize()
    assert torch.all(out[rows:] == mark)
    want = product64(a[:few], sa[:few], b[0], sb[0]).to(torch.bfloat16)
    for r in range(0, rows, max(few, rows // 64 // few * few)):
        got = out[r:r + few]
        assert torch.all((got == want) | (got == mark))


def test_quant_far_rows():
    M, N = 1_100_000, 2048
    x = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    row = torch.randn(7, 2 * N, generator=gen(3), device="cuda").bfloat16()
    x.zero_()
    x[-7:] = row
    say("quant far rows")
    q, s = fm.quant_fp8_blocks(x, gated=True)
    q0, s0 = fm.quant_fp8_blocks(row, gated=True)
    torch.cuda.synchronize()
    assert torch.equal(q[-7:], q0) and torch.equal(s[-7:], s0)
    assert not q[:100].any() and torch.all(s[:100] == 1)


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refusals():
    a, sa, b, sb = gemm_operands(gen(4), 8, 32, 256)
    ok = fm.gemm_fp8_blocks(a, sa, b, sb)
    assert torch.equal(ok, fm.gemm_fp8_blocks(a.view(torch.uint8), sa, b.view(torch.uint8), sb))
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, sa[:, :1].contiguous(), b, sb)
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, sa, b[:, :128].contiguous(), sb)
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, sa, b.t(), sb)
    with pytest.raises(TypeError):
        fm.gemm_fp8_blocks(a, sa, b, sb, out=torch.empty(8, 32, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        fm.gemm_fp8_blocks(a, sa.double(), b, sb)
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, sa, b, sb, out=torch.empty(8, 33, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fm.gemm_fp8_blocks(a, sa, b, sb, addend=ok[:4])
    with pytest.raises(fm.Fp8MoeError):
        fm.gemm_fp8_blocks(a, sa, b, sb, addend=ok, out=ok.view(-1).view(8, 32), out_dtype=torch.float32,
                           weight_layout=7)
    deep = gemm_operands(gen(5), 8, 32, 2048)
    with pytest.raises(fm.Fp8MoeError):      # a workspace below its size
        fm.gemm_fp8_blocks(*deep, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    ptr = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fm.grouped_gemm_fp8_ragged(a, sa, b[None], sb[None], ptr[:1])
    with pytest.raises(TypeError):
        fm.grouped_gemm_fp8_ragged(a, sa, b[None], sb[None], ptr.long())
    with pytest.raises(TypeError):
        fm.grouped_gemm_bf16_ragged(a, b[None], ptr)
    with pytest.raises(ValueError):
        fm.quant_fp8_blocks(torch.zeros(4, 129, device="cuda"), gated=True)
    with pytest.raises(fm.Fp8MoeError):
        fm.quant_fp8_blocks(torch.zeros(4, 24, device="cuda"))
    assert fm.gemm_fp8_blocks(a[:0], sa[:0], b, sb).shape == (0, 32)
    assert fm.quant_fp8_blocks(torch.zeros(0, 128, device="cuda"))[0].shape == (0, 128)
