"""Workloads of the products beside the routed layer: the dense FP8 product with block scales, the products grouped
by expert over ragged rows in FP8 and bf16, and the quantiser that makes their FP8 operands.

`listed()` names the cases, `draw(rng)` gives more of the same ranges, `prepare(case, seed)` makes a case's inputs
on the GPU, and `run(state)` is one pass: elementary torch operations where `own` is false, the library's entry
points where it is true.  `exact(case, seed)` computes the same outputs from the definitions in 64 bits, and
`work(case)` says what a pass cannot do without.

e4m3 codes come back as the values they stand for (torch's float8 type of the same bits).
"""

import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _gemm(M, N, K, addend=False, tiled=False):
    return {"op": "gemm", "M": M, "N": N, "K": K, "addend": addend, "tiled": tiled}


def _grouped(fmt, R, N, K, E, skew=0.0, spare=0, out="bf16", tiled=False):
    return {"op": "grouped", "fmt": fmt, "R": R, "N": N, "K": K, "E": E, "skew": skew, "spare": spare, "out": out,
            "tiled": tiled}


def _quant(M, N, gated=False, x="bf16"):
    return {"op": "quant", "M": M, "N": N, "gated": gated, "x": x}


def listed():
    return [
        # the down projection of one decoded token through a dense FFN or a shared expert: latency
        dict(_gemm(1, 7168, 2048, tiled=True), name="gemm M=1"),
        # a decode batch through a projection of odd width, weights as they were loaded
        dict(_gemm(33, 1500, 7168), name="gemm M=33"),
        # the shared expert's down projection of a short prefill, added to the routed experts' output
        dict(_gemm(512, 7168, 2048, addend=True, tiled=True), name="gemm addend M=512"),
        # ragged in every size: the last block of K holds 16 values, the last of N 80 rows
        dict(_gemm(1111, 2000, 1936), name="gemm ragged M=1111"),
        # a prefill chunk through gate and up of a dense FFN: the matrix cores' rate
        dict(_gemm(8192, 4096, 7168, tiled=True), name="gemm M=8192"),
        # 64 tokens' rows, sorted by expert, through gate and up of the large layer: a stream of weights
        dict(_grouped("fp8", 512, 4096, 7168, 256, tiled=True), name="grouped fp8 R=512"),
        # a prefill chunk's rows of very uneven popularity in a buffer for more of them
        dict(_grouped("fp8", 32768, 1536, 2048, 128, skew=1.2, spare=1024, tiled=True),
             name="grouped fp8 skewed R=32768"),
        # a prefill chunk's rows through the down projections of the large layer, weights as they were loaded
        dict(_grouped("fp8", 65536, 7168, 2048, 256), name="grouped fp8 R=65536"),
        # a small decode batch through unquantised experts
        dict(_grouped("bf16", 264, 1536, 2048, 128, skew=1.2, tiled=True), name="grouped bf16 R=264"),
        # a prefill chunk's rows through unquantised down projections
        dict(_grouped("bf16", 32768, 2048, 768, 128, skew=1.2), name="grouped bf16 skewed R=32768"),
        # the activations of one decoded token ahead of a projection: latency
        dict(_quant(1, 7168), name="quant M=1"),
        # SwiGLU and quantisation between the grouped products of a prefill chunk: a stream through HBM
        dict(_quant(65536, 2048, gated=True), name="quant gated M=65536"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "grouped", "grouped", "quant"])
    if op == "quant":
        M, gated = _log(rng, 1, 32768), rng.random() < 0.5
        return _quant(M, 16 * _log(rng, 1, 128 if gated else 448), gated, rng.choice(["bf16", "bf16", "f32"]))
    tiled = rng.random() < 0.5
    if op == "gemm":
        N, K = _log(rng, 8, 7168), 16 * _log(rng, 1, 448)
        if tiled:       # the tiled layout holds whole bands of 16 rows and blocks of 128 bytes
            N, K = -(-N // 16) * 16, -(-K // 128) * 128
        return _gemm(_log(rng, 1, 8192), N, K, rng.random() < 0.3, tiled)
    fmt = rng.choice(["fp8", "bf16"])
    N, K = _log(rng, 16, 4096), 16 * _log(rng, 2, 256 if fmt == "fp8" else 128)
    if tiled:
        N, K = -(-N // 16) * 16, -(-K // 128) * 128
    return _grouped(fmt, _log(rng, 1, 32768), N, K, _log(rng, 1, 160), rng.choice([0.0, 1.2]),
                    rng.choice([0, 0, 100]), "f32" if fmt == "bf16" and rng.random() < 0.3 else "bf16", tiled)


# ---------------------------------------------------------------- inputs

def _blocks(n):
    return -(-n // BLOCK)


def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + tag) & ((1 << 62) - 1))
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _activations(g, M, K):
    """Normally distributed rows with a few channels far larger than the rest."""
    return _randn(g, M, K).mul_(1 + 20 * (torch.rand(K, generator=g, device=DEV) < 0.01))


def _fp8_rows(g, M, K):
    """e4m3 rows with one scale per 128 columns, the largest value of a block at 448."""
    a = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(M, _blocks(K), device=DEV)
    for r in range(0, M, 16384):
        x = _activations(g, min(16384, M - r), K)
        pad = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(x.shape[0], -1, BLOCK)
        s = pad.abs().amax(2) / E4M3_MAX
        scale[r:r + 16384] = s
        a[r:r + 16384] = (pad / s[:, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).view(x.shape[0], -1)[:, :K].to(a.dtype)
    return a, scale


def _fp8_weights(g, E, N, K):
    """e4m3 codes of normally distributed weights, the largest of a block near 448, and scales per 128 x 128 that
    bring them to a spread of about 0.02."""
    w = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    for e in range(0, E, 16):
        n = min(16, E - e)
        w[e:e + n] = _randn(g, n, N, K, dtype=torch.float16).mul_(100).clamp_(-E4M3_MAX, E4M3_MAX).to(w.dtype)
    return w, torch.rand(E, _blocks(N), _blocks(K), generator=g, device=DEV) * 1e-4 + 1.5e-4


def _bf16_weights(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    for e in range(0, E, 16):
        n = min(16, E - e)
        w[e:e + n] = _randn(g, n, N, K, dtype=torch.bfloat16).mul_(0.02)
    return w


def _tile(w):
    """Row-major [E, N, K] -> the MFMA-tiled byte order that moe_pack_weights documents."""
    b = w.view(torch.uint8)
    E, N, K = b.shape
    b = b.view(E, N // 16, 16, K // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6).contiguous().view(E, N, K)
    return b.view(w.dtype)


def _group_sizes(case, seed):
    """Rows of each group: every row draws its group by popularity, the groups in an order of the seed's."""
    g = torch.Generator()
    g.manual_seed((int(seed) * 1000003 + 7) & ((1 << 62) - 1))
    E = case["E"]
    p = torch.arange(1, E + 1, dtype=torch.float64) ** -case["skew"]
    p = p[torch.randperm(E, generator=g)]
    return torch.bincount(torch.multinomial(p, case["R"], replacement=True, generator=g), minlength=E)


def prepare(case, seed):
    c = case
    g = _gen(seed, {"gemm": 1, "grouped": 2, "quant": 3}[c["op"]])
    s = {"case": dict(c)}
    if c["op"] == "quant":
        s["x"] = _activations(g, c["M"], (2 if c["gated"] else 1) * c["N"])
        if c["x"] == "bf16":
            s["x"] = s["x"].to(torch.bfloat16)
        return s
    if c["op"] == "gemm":
        s["a"], s["a_scale"] = _fp8_rows(g, c["M"], c["K"])
        w, scale = _fp8_weights(g, 1, c["N"], c["K"])
        s["b"], s["b_scale"] = w[0], scale[0]
        if c["tiled"]:      # laid out once, where the weights are loaded
            s["b_tiled"] = _tile(w)[0]
        s["addend"] = _randn(g, c["M"], c["N"]).to(torch.bfloat16) if c["addend"] else None
        return s
    sizes = _group_sizes(c, seed)
    s["sizes"] = sizes.tolist()
    s["m_indptr"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).to(DEV)
    rows = c["R"] + c["spare"]
    if c["fmt"] == "fp8":
        s["a"], s["a_scale"] = _fp8_rows(g, rows, c["K"])
        s["b"], s["b_scale"] = _fp8_weights(g, c["E"], c["N"], c["K"])
    else:
        s["a"] = _activations(g, rows, c["K"]).to(torch.bfloat16)
        s["b"] = _bf16_weights(g, c["E"], c["N"], c["K"])
    if c["tiled"]:
        s["b_tiled"] = _tile(s["b"])
    # rows behind the last group keep what the caller's buffer holds
    s["out"] = torch.zeros(rows, c["N"], dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _decode_rows(a, scale):
    return a.float() * scale.repeat_interleave(BLOCK, 1)[:, :a.shape[1]]


def _decode_weights(b, scale):
    N, K = b.shape
    return b.float() * scale.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _plain_gemm(s):
    y = _decode_rows(s["a"], s["a_scale"]) @ _decode_weights(s["b"], s["b_scale"]).t()
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return {"out": y.to(torch.bfloat16)}


def _plain_grouped(s):
    out, at = s["out"], 0
    for e, n in enumerate(s["sizes"]):
        if not n:
            continue
        a = s["a"][at:at + n]
        if s["case"]["fmt"] == "fp8":
            y = _decode_rows(a, s["a_scale"][at:at + n]) @ _decode_weights(s["b"][e], s["b_scale"][e]).t()
        else:
            y = a.float() @ s["b"][e].float().t()
        out[at:at + n] = y
        at += n
    return {"out": out}


def _plain_quant(s):
    v = s["x"].float()
    if s["case"]["gated"]:
        gate, up = v.chunk(2, dim=1)
        v = gate / (1 + torch.exp(-gate)) * up
    M, N = v.shape
    b = torch.nn.functional.pad(v, (0, _blocks(N) * BLOCK - N)).view(M, -1, BLOCK)
    amax = b.abs().amax(2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    q = (b / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(M, -1)[:, :N]
    return {"q": q.to(torch.float8_e4m3fn).contiguous(), "scale": scale}


# ---------------------------------------------------------------- the library's calls
#
# A state's first pass allocates its outputs and workspace, and the later ones write into the same buffers, as a
# serving loop does.

def _layout(fm, case):
    return fm.WEIGHTS_MFMA_TILED if case["tiled"] else fm.WEIGHTS_ROW_MAJOR


def _own_gemm(s):
    import fp8_block_scaled_moe_amd as fm
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = fm.alloc_workspace_gemm(c["M"], c["N"], c["K"], s["a"].device)
    s["kept"] = fm.gemm_fp8_blocks(s["a"], s["a_scale"], s["b_tiled" if c["tiled"] else "b"], s["b_scale"],
                                   addend=s["addend"], out=s.get("kept"), workspace=s["workspace"],
                                   weight_layout=_layout(fm, c))
    return {"out": s["kept"]}


def _own_grouped(s):
    import fp8_block_scaled_moe_amd as fm
    c = s["case"]
    b = s["b_tiled" if c["tiled"] else "b"]
    if c["fmt"] == "fp8":
        out = fm.grouped_gemm_fp8_ragged(s["a"], s["a_scale"], b, s["b_scale"], s["m_indptr"], out=s["out"],
                                         weight_layout=_layout(fm, c))
    else:
        out = fm.grouped_gemm_bf16_ragged(s["a"], b, s["m_indptr"], out=s["out"], weight_layout=_layout(fm, c))
    return {"out": out}


def _own_quant(s):
    import fp8_block_scaled_moe_amd as fm
    q, scale = s.get("kept", (None, None))
    q, scale = s["kept"] = fm.quant_fp8_blocks(s["x"], gated=s["case"]["gated"], q=q, scale=scale)
    return {"q": q.view(torch.float8_e4m3fn), "scale": scale}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gemm": _own_gemm, "grouped": _own_grouped, "quant": _own_quant}[op](state)
    return {"gemm": _plain_gemm, "grouped": _plain_grouped, "quant": _plain_quant}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _active_groups(case):
    """Groups that get a row, as expected from their popularity."""
    p = [(e + 1) ** -case["skew"] for e in range(case["E"])]
    total = sum(p)
    return sum(1 - (1 - v / total) ** case["R"] for v in p)


def work(case):
    c = case
    N = c["N"]
    if c["op"] == "quant":
        x = (2 if c["gated"] else 1) * (2 if c["x"] == "bf16" else 4)
        return {"bytes": c["M"] * (x * N + N + 4 * _blocks(N)), "flops": (10 if c["gated"] else 4) * c["M"] * N}
    K = c["K"]
    if c["op"] == "gemm":
        M = c["M"]
        return {"bytes": (M + N) * K + 4 * (M + _blocks(N)) * _blocks(K) + (4 if c["addend"] else 2) * M * N,
                "flops": 2 * M * N * K}
    row = K + 4 * _blocks(K) if c["fmt"] == "fp8" else 2 * K
    weights = N * K + 4 * _blocks(N) * _blocks(K) if c["fmt"] == "fp8" else 2 * N * K
    out = (4 if c["out"] == "f32" else 2) * N
    return {"bytes": int(c["R"] * (row + out) + _active_groups(c) * weights + 4 * (c["E"] + 1)),
            "flops": 2 * c["R"] * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits

def _product64(a, a_scale, b, b_scale):
    """Block by block of the contraction: the codes' sums, then their scales."""
    M, K = a.shape
    N = b.shape[0]
    if a_scale is None:
        return a.double() @ b.double().t()
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    row = torch.arange(N, device=DEV) // BLOCK
    for k in range(_blocks(K)):
        cut = slice(k * BLOCK, min((k + 1) * BLOCK, K))
        p = a[:, cut].double() @ b[:, cut].double().t()
        y += p * a_scale[:, k].double()[:, None] * b_scale[row, k].double()
    return y


def _exact_gemm(s):
    y = _product64(s["a"], s["a_scale"], s["b"], s["b_scale"])
    return {"out": y if s["addend"] is None else y + s["addend"].double()}


def _exact_grouped(s):
    c = s["case"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    ends = s["m_indptr"].tolist()
    fp8 = c["fmt"] == "fp8"
    for e in range(c["E"]):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            out[lo:hi] = _product64(s["a"][lo:hi], s["a_scale"][lo:hi] if fp8 else None, s["b"][e],
                                    s["b_scale"][e] if fp8 else None)
    return {"out": out}


def _exact_quant(s):
    c, v = s["case"], s["x"].double()
    M, N = c["M"], c["N"]
    if c["gated"]:
        gate = v[:, :N]
        v = gate * torch.sigmoid(gate) * v[:, N:]
    # the values ahead of their rounding to the output's type, as for every other output
    q, scale = torch.empty_like(v), torch.ones(M, _blocks(N), dtype=torch.float64, device=DEV)
    for k in range(_blocks(N)):
        cut = slice(k * BLOCK, min((k + 1) * BLOCK, N))
        amax = v[:, cut].abs().amax(1)
        scale[:, k] = torch.where(amax > 0, amax / E4M3_MAX, scale[:, k])
        q[:, cut] = v[:, cut] / scale[:, k, None]
    return {"q": q, "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemm": _exact_gemm, "grouped": _exact_grouped, "quant": _exact_quant}[case["op"]](s)
