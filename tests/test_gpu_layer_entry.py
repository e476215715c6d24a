"""The layer's entry as a model runs it: residual addition and norm, the router on the norm's bf16 output, and the
experts on its quantised one, in every format the norm makes, from one token to a prefill chunk.

Each step is held to its oracle on the inputs the GPU gave it; the whole is captured into a graph and replayed.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
import synth
from oracle import int8 as O8
from oracle import moe as OM
from oracle.norm import add_rmsnorm_reference
from oracle.router import router_reference
from tests.gpu_helpers import assert_rows_close_to_oracle, say

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 256, 16, 4


class Entry:
    """One layer's weights and its call, every buffer preallocated."""

    def __init__(self, T, fmt, seed=0):
        self.T, self.fmt = T, fmt
        g = torch.Generator().manual_seed(seed)
        self.norm_w = (1 + 0.2 * torch.randn(H, generator=g)).bfloat16().cuda()
        self.gate = (torch.randn(E, H, generator=g) / H ** 0.5).bfloat16().cuda()
        self.bias = (0.1 * torch.randn(E, generator=g)).cuda()
        if fmt == "int8":
            self.w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, dtype=torch.int8).cuda()
            self.w2 = torch.randint(-127, 128, (E, H, I), generator=g, dtype=torch.int8).cuda()
            self.w13s = (torch.rand(E, 2 * I, generator=g) + 0.5).cuda() * 0.02 / H ** 0.5
            self.w2s = (torch.rand(E, H, generator=g) + 0.5).cuda() * 0.02 / I ** 0.5
        elif fmt == "fp8":
            self.w13, self.w13s = synth.expert_weight_set(E, 2 * I, H, 9, synth.TAG_W13, device="cuda")
            self.w2, self.w2s = synth.expert_weight_set(E, H, I, 9, synth.TAG_W2, device="cuda")
        else:
            self.w13, self.w13s = synth.expert_weight_set_mx(E, 2 * I, H, 9, synth.TAG_W13, device="cuda")
            self.w2, self.w2s = synth.expert_weight_set_mx(E, H, I, 9, synth.TAG_W2, device="cuda")
        self.x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        self.res = torch.empty(T, H, dtype=torch.float32, device="cuda")
        self.fill(seed)
        alloc = {"int8": fm.alloc_workspace_int8, "fp8": fm.alloc_workspace, "mxfp8": fm.alloc_workspace_mx}[fmt]
        self.ws = alloc(T, H, I, E, K, "cuda")
        self.norm_fmt = {"int8": fm.NORM_INT8, "fp8": fm.NORM_FP8, "mxfp8": fm.NORM_MXFP8}[fmt]
        self.fused = {"int8": fm.moe_fused_int8, "fp8": fm.moe_fused_fp8, "mxfp8": fm.moe_fused_mxfp8}[fmt]

    def fill(self, seed):
        g = torch.Generator().manual_seed(100 + seed)
        self.x.copy_(torch.randn(self.T, H, generator=g))
        self.res.copy_(3 * torch.randn(self.T, H, generator=g))

    def __call__(self):
        q, s, n, v = fm.add_rmsnorm_quant(self.x, self.norm_w, 1e-6, self.norm_fmt, residual=self.res, want_norm=True)
        logits = torch.matmul(n.float(), self.gate.float().t())
        ids, w = fm.moe_router_topk(logits, K, fm.SCORE_SIGMOID, bias=self.bias, n_group=4, topk_group=2, group_top=2,
                                    scale=2.5)
        out = self.fused(q, s, self.w13, self.w13s, self.w2, self.w2s, ids, w, workspace=self.ws)
        return q, s, n, v, logits, ids, w, out


@pytest.mark.parametrize("fmt", ["int8", "fp8", "mxfp8"])
@pytest.mark.parametrize("T", [1, 3, 37, 515])
def test_entry(T, fmt):
    say("layer entry", fmt, T)
    e = Entry(T, fmt, seed=T)
    q, s, n, v, logits, ids, w, out = e()
    torch.cuda.synchronize()
    c = lambda t: t.cpu().numpy()
    vr, nr = add_rmsnorm_reference(e.x.cpu().double().numpy(), c(e.res), e.norm_w.cpu().double().numpy(), 1e-6, False)
    assert np.array_equal(c(v).astype(np.float64), vr)
    assert np.all(np.abs(n.cpu().double().numpy() - nr) <= np.abs(nr) * (2.0 ** -8 + 96 * 2.0 ** -24))
    rid, rw = router_reference(c(logits), K, "sigmoid", c(e.bias), 4, 2, 2, True, 2.5)
    assert np.array_equal(c(ids), rid) and np.allclose(c(w), rw, rtol=4e-6)
    if fmt == "int8":
        ref = O8.moe_reference_int8(c(q), c(s), c(e.w13), c(e.w13s), c(e.w2), c(e.w2s), c(ids), c(w))
    else:
        f = OM.moe_reference if fmt == "fp8" else OM.moe_reference_mx
        ref = f(c(q), c(s), c(e.w13), c(e.w13s), c(e.w2), c(e.w2s), c(ids), c(w))[1]
    assert_rows_close_to_oracle(out, ref, f"layer entry {fmt} T={T}")


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T", [1, 64])
def test_entry_in_a_graph(T, fmt):
    say("layer entry graph", fmt, T)
    e = Entry(T, fmt)
    e()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = e()
    for seed in (1, 2, 3):
        e.fill(seed)
        g.replay()
        torch.cuda.synchronize()
        want = e()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    """Two calls at once, each with its own workspace."""
    a, b = Entry(200, "int8", 1), Entry(200, "int8", 2)
    want = a()[-1].clone(), b()[-1].clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            ra = a()[-1]
        with torch.cuda.stream(sb):
            rb = b()[-1]
        sa.synchronize()
        sb.synchronize()
        assert torch.equal(ra, want[0]) and torch.equal(rb, want[1])
