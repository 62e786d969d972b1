"""The experts' products in 8-bit floating point, as they are measured.

Five operators that stand between the dispatch and the combine of a mixture of
experts: the quantisation to 8 bits with a scale for each block of 128 (quant),
the experts' activation with its gradient, quantised where it is formed
(swiglu), the grouped product of the sorted rows with their experts' weights
(gemm), the weights' gradient (wgrad), and the whole layer for a few tokens
(few).  `own` chooses between the library's calls and the same mathematics in
elementary torch operations, in fp32 and rounded once.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128
LEAST = 2.0 ** -100  # a block's largest magnitude counts as no less


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the rows of a small serving batch on their way into a product
        {"name": "quant_batch", "op": "quant", "R": 37, "C": 7168, "G": 1, "mode": "rows",
         "dtype": "fp16", "fmt": "e4m3"},
        # the sorted rows of a training step, along C for the product, along the rows for the
        # weights' gradient
        {"name": "quant_layer", "op": "quant", "R": 73664, "C": 4096, "G": 1, "mode": "both",
         "dtype": "bf16", "fmt": "e4m3"},
        # the experts' activation in a training step
        {"name": "swiglu_fwd_layer", "op": "swiglu", "way": "fwd", "R": 73664, "F": 2048,
         "mode": "both", "dtype": "bf16", "fmt": "e4m3"},
        # its gradient, in the wider-ranged format, odd sizes
        {"name": "swiglu_bwd_ragged", "op": "swiglu", "way": "bwd", "R": 9136, "F": 1328,
         "mode": "both", "dtype": "bf16", "fmt": "e5m2"},
        # gate and up product of a serving batch: few rows an expert, segments off the tiles
        {"name": "gemm_batch", "op": "gemm", "S": 296, "E": 60, "align": 8, "N": 2816, "K": 4096,
         "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # gate and up product of a training step
        {"name": "gemm_layer", "op": "gemm", "S": 65536, "E": 64, "align": 128, "N": 4096,
         "K": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # the gradient on its way back through an odd down product, in the wider-ranged format
        {"name": "gemm_grad_ragged", "op": "gemm", "S": 7001, "E": 61, "align": 16, "N": 1328,
         "K": 7168, "a": "e5m2", "b": "e4m3", "out": "fp16"},
        # the weights' gradient of a training step
        {"name": "wgrad_layer", "op": "wgrad", "S": 65536, "E": 64, "align": 128, "M": 4096,
         "N": 2048, "a": "e5m2", "b": "e4m3", "out": "fp32"},
        # a small step over many experts, some of them without a row, odd sizes
        {"name": "wgrad_ragged", "op": "wgrad", "S": 3001, "E": 61, "align": 128, "M": 1000,
         "N": 1328, "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # one new token of one sequence while serving the wide model, weights in 8 bits
        {"name": "few_token", "op": "few", "T": 1, "C": 7168, "F": 2048, "E": 64, "k": 8,
         "dtype": "bf16", "weights": "e4m3"},
        # a small serving batch, weights in 16 bits
        {"name": "few_batch", "op": "few", "T": 13, "C": 4096, "F": 1408, "E": 60, "k": 4,
         "dtype": "bf16", "weights": "bf16"},
        # a larger one, odd sizes, weights in 8 bits
        {"name": "few_tokens", "op": "few", "T": 64, "C": 2896, "F": 2000, "E": 128, "k": 6,
         "dtype": "fp16", "weights": "e4m3"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "swiglu", "gemm", "gemm", "wgrad", "few", "few"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op in ("quant", "swiglu"):
        mode = rng.choice(["rows", "both", "both", "columns", "tiles"][:5 if op == "quant" else 4])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        C = 16 * _log_int(rng, 8, 512)
        R = _log_int(rng, 1, 73664)
        while R > 1 and R * C > 300_000_000 // (2 if dtype == "fp32" else 1):
            R = (R + 1) // 2
        if mode != "rows":
            R = (R + 15) // 16 * 16
        if op == "quant":
            G = rng.choice([1, 3, 8]) if mode == "tiles" and R <= 8192 else 1
            return {"op": op, "R": R, "C": C, "G": G, "mode": mode, "dtype": dtype, "fmt": fmt}
        return {"op": op, "way": rng.choice(["fwd", "bwd"]), "R": R, "F": max(64, C // 2 // 16 * 16),
                "mode": mode, "dtype": dtype, "fmt": fmt}
    if op == "few":
        T, E = _log_int(rng, 1, 64), _log_int(rng, 4, 256)
        C, F = 16 * _log_int(rng, 16, 448), 16 * _log_int(rng, 16, 256)
        while E > 4 and E * 3 * C * F > 2_800_000_000:
            E = (E + 1) // 2
        dtype = rng.choice(["bf16", "fp16"])
        return {"op": op, "T": T, "C": C, "F": F, "E": E, "k": min(E, rng.randint(1, 8)),
                "dtype": dtype, "weights": rng.choice(["e4m3", "e4m3", dtype])}
    S, E = _log_int(rng, 1, 65536), _log_int(rng, 1, 256)
    if op == "gemm":
        N, K = 8 * _log_int(rng, 16, 900), 16 * _log_int(rng, 8, 448)
        while E > 1 and E * N * K > 1_100_000_000:
            E = (E + 1) // 2
        while S * N * K > 1_100_000_000_000:
            S = (S + 1) // 2
        return {"op": op, "S": S, "E": E, "align": rng.choice([1, 16, 128, 128]), "N": N, "K": K,
                "a": fmt, "b": "e4m3", "out": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    M, N = 8 * _log_int(rng, 16, 900), 8 * _log_int(rng, 16, 900)
    while E > 1 and E * M * N > 540_000_000:
        E = (E + 1) // 2
    while S * M * N > 540_000_000_000:
        S = (S + 1) // 2
    return {"op": op, "S": S, "E": E, "align": 128, "M": M, "N": N, "a": fmt, "b": "e4m3",
            "out": rng.choice(["fp32", "fp32", "bf16"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(g, R, C):
    """Rows of a size of their own, a few channels far larger than the others."""
    x = _randn(g, R, C)
    x *= 0.25 + 2 * _rand(g, R, 1)
    x *= 1 + 20 * (_rand(g, C) < 0.004)
    return x


def _weights(g, E, N, K, fmt):
    """Experts' weights and their scales, an expert at a time."""
    q = _empty(E, N, K, dtype=DTYPES[fmt])
    s = _empty(E, _blocks(K), _blocks(N))
    for e in range(E):
        q[e], s[e] = _quant_tiles(_randn(g, N, K) * K ** -0.5, fmt)
    return q, s


def _segments(g, S, E, align):
    """Rows of each expert, their segments' starts in tiles of `align` rows; some experts are
    more popular, and some have no row where there are few."""
    popular = 0.5 + _rand(g, E)
    pick = torch.multinomial(popular, S, replacement=True, generator=g)
    counts = torch.bincount(pick, minlength=E)
    tiles = (counts + align - 1) // align * align
    offsets = torch.cat((torch.zeros_like(tiles[:1]), tiles.cumsum(0)))
    return counts, offsets.int(), int(tiles.max())


def _sorted_rows(S, E, align):
    """Rows that are allocated for the sorted slots, in whole blocks."""
    return _blocks(S + min(E, S) * (align - 1)) * BLOCK


def _with_padding(x, counts, offsets):
    """Rows without a slot hold zeros, as the dispatch leaves them."""
    r = torch.arange(x.shape[0], device=x.device)
    e = (torch.searchsorted(offsets.long(), r, right=True) - 1).clamp(0, counts.shape[0] - 1)
    return torch.where((r - offsets[e] < counts[e])[:, None], x, torch.zeros_like(x))


def _outputs_of_quant(s, G, R, C, mode, fmt):
    lead, dt = (G,) if G > 1 else (), DTYPES[fmt]
    tiles = mode == "tiles"
    s["q"] = s["s"] = s["qt"] = s["st"] = None
    if mode != "columns":
        s["q"] = _empty(*lead, R, C, dtype=dt)
        s["s"] = _empty(*lead, _blocks(C), _blocks(R) if tiles else R)
    if mode != "rows":
        s["qt"] = _empty(*lead, C, R, dtype=dt)
        s["st"] = _empty(*lead, _blocks(R), _blocks(C) if tiles else C)


def prepare(case, seed):
    g = _generator(seed)
    s, op = {"case": case}, case["op"]
    if op == "quant":
        G, R, C, mode = (case[n] for n in ("G", "R", "C", "mode"))
        x = _activations(g, G * R, C).to(DTYPES[case["dtype"]])
        s["x"] = x.reshape(G, R, C) if G > 1 else x
        _outputs_of_quant(s, G, R, C, mode, case["fmt"])
        return s
    if op == "swiglu":
        R, F, dt = case["R"], case["F"], DTYPES[case["dtype"]]
        s["h"] = _activations(g, R, 2 * F).to(dt)
        if case["way"] == "bwd":
            s["da"] = (0.1 * _activations(g, R, F)).to(dt)
        _outputs_of_quant(s, 1, R, F if case["way"] == "fwd" else 2 * F, case["mode"], case["fmt"])
        return s
    if op == "few":
        T, C, F, E, k = (case[n] for n in ("T", "C", "F", "E", "k"))
        dt, fmt = DTYPES[case["dtype"]], case["weights"]
        s["x"] = _activations(g, T, C).to(dt)
        popular = torch.log(_rand(g, E) + 0.05)
        noise = -torch.log(-torch.log(_rand(g, T, E) * 0.9998 + 1e-4))
        ids = torch.topk(popular + noise, k, dim=1).indices.int()
        s["ids"] = torch.where(_rand(g, T, k) < 1 / 64, torch.full_like(ids, -1), ids).contiguous()
        w = _rand(g, T, k) + 0.02
        s["w"] = w / w.sum(1, keepdim=True)
        s["s1"] = s["s2"] = None
        if fmt == "e4m3":
            s["w1"], s["s1"] = _weights(g, E, 2 * F, C, fmt)
            s["w2"], s["s2"] = _weights(g, E, C, F, fmt)
        else:
            s["w1"], s["w2"] = _empty(E, 2 * F, C, dtype=dt), _empty(E, C, F, dtype=dt)
            for e in range(E):
                s["w1"][e] = _randn(g, 2 * F, C) * C ** -0.5
                s["w2"][e] = _randn(g, C, F) * F ** -0.5
        s["f"] = _empty(T, C, dtype=dt)
        return s
    S, E, align = case["S"], case["E"], case["align"]
    counts, s["offsets"], s["cap"] = _segments(g, S, E, align)
    R = _sorted_rows(S, E, align)
    if op == "gemm":
        N, K = case["N"], case["K"]
        x = _with_padding(_activations(g, R, K), counts, s["offsets"])
        s["a"], s["sa"] = _quant_rows(x, case["a"])
        s["b"], s["sb"] = _weights(g, E, N, K, case["b"])
        s["out"] = _empty(R, N, dtype=DTYPES[case["out"]])
        return s
    M, N = case["M"], case["N"]
    s["at"], s["sat"] = _quant_columns(_with_padding(0.1 * _activations(g, R, M), counts,
                                                     s["offsets"]), case["a"])
    s["bt"], s["sbt"] = _quant_columns(_with_padding(_activations(g, R, N), counts, s["offsets"]),
                                       case["b"])
    s["out"] = _empty(E, M, N, dtype=DTYPES[case["out"]])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _padded(x, dim):
    """Zeros after the last of `dim` up to whole blocks."""
    more = -x.shape[dim] % BLOCK
    if not more:
        return x
    shape = list(x.shape)
    shape[dim] = more
    return torch.cat((x, x.new_zeros(shape)), dim)


def _scale(amax, fmt):
    """A block's scale and what its values are multiplied by, both IEEE quotients.  A block with
    an infinity or a NaN has the scale NaN."""
    amax = amax.clamp(min=LEAST)
    top = torch.full_like(amax, LARGEST[fmt])
    return torch.where(amax.isfinite(), amax / top, math.nan), top / amax


def _quant_rows(x, fmt):
    """x [..., R, C] fp32: q [..., R, C] and s [..., blocks of C, R]."""
    p = _padded(x, -1).unflatten(-1, (-1, BLOCK))
    s, up = _scale(p.abs().amax(-1), fmt)
    q = (p * up[..., None]).flatten(-2)[..., :x.shape[-1]].to(DTYPES[fmt])
    return q.contiguous(), s.transpose(-1, -2).contiguous()


def _quant_columns(x, fmt):
    """x [..., R, C] fp32: qt [..., C, R] and st [..., blocks of R, C]."""
    return _quant_rows(x.transpose(-1, -2).contiguous(), fmt)


def _quant_tiles(x, fmt):
    """x [..., R, C] fp32: q [..., R, C] and s [..., blocks of C, blocks of R]."""
    p = _padded(_padded(x, -1), -2).unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    s, up = _scale(p.abs().amax((-1, -3)), fmt)
    q = (p * up[..., :, None, :, None]).flatten(-2).flatten(-3, -2)
    q = q[..., :x.shape[-2], :x.shape[-1]].to(DTYPES[fmt])
    return q.contiguous(), s.transpose(-1, -2).contiguous()


def _plain_quant(x, mode, fmt):
    out = {}
    if mode == "tiles":
        q, s = _quant_tiles(x, fmt)
        return {"q": q, "s": s, "qt": q.transpose(-1, -2).contiguous(),
                "st": s.transpose(-1, -2).contiguous()}
    if mode != "columns":
        out["q"], out["s"] = _quant_rows(x, fmt)
    if mode != "rows":
        out["qt"], out["st"] = _quant_columns(x, fmt)
    return out


def _swiglu(h):
    g, u = h.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _swiglu_grad(da, h):
    g, u = h.chunk(2, -1)
    p = 1 / (1 + torch.exp(-g))
    return torch.cat((da * u * p * (1 + g * (1 - p)), da * g * p), -1)


def _values(q, s):
    """The rows q [..., R, K] as they stand for, s [..., blocks of K, R or blocks of R]."""
    s = s.transpose(-1, -2)
    if s.shape[-2] != q.shape[-2]:
        s = s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _by_expert(offsets, cap, R):
    """[E, cap]: the rows of each expert's segment, R behind its end; [R]: a row's place in
    that, E*cap for the rows past the last segment."""
    E = offsets.shape[0] - 1
    first = offsets[:-1].long()[:, None]
    rows = first + torch.arange(cap, device=offsets.device)
    at = torch.where(rows < offsets[1:].long()[:, None], rows, torch.full_like(rows, R))
    place = torch.full((R + 1,), E * cap, device=offsets.device)
    place.scatter_(0, at.reshape(-1), torch.arange(E * cap, device=offsets.device))
    return at, place[:R]


def _plain_gemm(a, sa, b, sb, offsets, cap, dtype):
    at, place = _by_expert(offsets, cap, a.shape[0])
    rows = torch.cat((_values(a, sa), sa.new_zeros(1, a.shape[1])))[at]
    y = torch.bmm(rows, _values(b, sb).transpose(1, 2)).flatten(0, 1)
    # a row past the last segment takes none of them
    kept = (place < y.shape[0])[:, None]
    return torch.where(kept, y[place.clamp(max=y.shape[0] - 1)], y.new_zeros(())).to(dtype)


def _plain_wgrad(at, sat, bt, sbt, offsets, cap, dtype):
    rows, _ = _by_expert(offsets, cap, at.shape[1])
    a = torch.cat((_values(at, sat).t(), sat.new_zeros(1, at.shape[0])))[rows]
    b = torch.cat((_values(bt, sbt).t(), sbt.new_zeros(1, bt.shape[0])))[rows]
    return torch.bmm(a.transpose(1, 2), b).to(dtype)


def _rounded(x, fmt):
    """x [..., C] as its blocks of 128 stand for it after their quantisation."""
    p = _padded(x, -1).unflatten(-1, (-1, BLOCK))
    s, up = _scale(p.abs().amax(-1, keepdim=True), fmt)
    return ((p * up).to(DTYPES[fmt]).float() * s).flatten(-2)[..., :x.shape[-1]]


def _plain_few(s):
    x, ids, w = s["x"].float(), s["ids"].long(), s["w"]
    (T, k), E = ids.shape, s["w1"].shape[0]
    kept, at = ids >= 0, ids.clamp(min=0)
    eight = s["s1"] is not None
    if eight:
        x = _rounded(x, "e4m3")

    def weights(name, scales, of):
        q = s[name][of] if of is not None else s[name]
        if not eight:
            return q.float()
        return _values(q, s[scales][of] if of is not None else s[scales])

    if T * k < E:  # the weights of each slot's expert
        of, rows = at.reshape(-1), x.repeat_interleave(k, 0)[:, None]
    else:  # every token with every expert
        of, rows = None, x[None].expand(E, T, -1)
    a = _swiglu(torch.bmm(rows, weights("w1", "s1", of).transpose(1, 2)))
    if eight:
        a = _rounded(a, "e4m3")
    y = torch.bmm(a, weights("w2", "s2", of).transpose(1, 2))
    if of is not None:
        y = y.reshape(T, k, -1)
    else:
        y = y[at, torch.arange(T, device=x.device)[:, None]]
    y = torch.where(kept[..., None], w[..., None] * y, y.new_zeros(()))
    return y.sum(1).to(s["x"].dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quant":
        return _plain_quant(s["x"].float(), c["mode"], c["fmt"])
    if op == "swiglu" and c["way"] == "fwd":
        return _plain_quant(_swiglu(s["h"].float()), c["mode"], c["fmt"])
    if op == "swiglu":
        return _plain_quant(_swiglu_grad(s["da"].float(), s["h"].float()), c["mode"], c["fmt"])
    if op == "gemm":
        return {"out": _plain_gemm(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["cap"],
                                   s["out"].dtype)}
    if op == "wgrad":
        return {"out": _plain_wgrad(s["at"], s["sat"], s["bt"], s["sbt"], s["offsets"], s["cap"],
                                    s["out"].dtype)}
    return {"f": _plain_few(s)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import layers_proj_rms_gb300 as M
    c = s["case"]
    op = c["op"]
    if op in ("quant", "swiglu"):
        outs = (s["q"], s["s"], s["qt"], s["st"])
        if op == "quant":
            M.mhc_fp8_quant(s["x"], *outs, tiles=c["mode"] == "tiles")
        elif c["way"] == "fwd":
            M.mhc_fp8_swiglu_fwd(s["h"], None, *outs)
        else:
            M.mhc_fp8_swiglu_bwd(s["da"], s["h"], None, *outs)
        return {n: s[n] for n in ("q", "s", "qt", "st") if s[n] is not None}
    if op == "gemm":
        M.mhc_fp8_gemm(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["out"])
        return {"out": s["out"]}
    if op == "wgrad":
        M.mhc_fp8_wgrad(s["at"], s["sat"], s["bt"], s["sbt"], s["offsets"], s["out"])
        return {"out": s["out"]}
    if "ws" not in s:
        s["ws"] = M.workspace(M.OP_MOE_FEW_FWD, c["T"], c["k"], c["C"] + c["F"])
    M.mhc_moe_few_fwd(s["x"], s["ids"], s["w"], s["w1"], s["w2"], s["f"], s["ws"], s["s1"],
                      s["s2"])
    return {"f": s["f"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("quant", "swiglu"):
        b, mode, R = DTYPES[case["dtype"]].itemsize, case["mode"], case["R"]
        if op == "quant":
            C, read = case["C"], case["G"] * R * case["C"]
            out = read
        else:
            C = case["F"] * (1 if case["way"] == "fwd" else 2)
            read, out = R * case["F"] * (2 if case["way"] == "fwd" else 3), R * C
        once = {"rows": out // BLOCK, "columns": out // BLOCK, "both": out // BLOCK,
                "tiles": out // BLOCK ** 2}[mode]
        both = 2 if mode in ("both", "tiles") else 1
        flops = {"quant": 3, "swiglu": 10}[op]
        return {"bytes": read * b + both * (out + 4 * once), "flops": flops * out}
    if op == "gemm":
        S, E, N, K = (case[n] for n in ("S", "E", "N", "K"))
        b = DTYPES[case["out"]].itemsize
        used = E * (1 - (1 - 1 / E) ** S)  # experts with a row, on average
        R = _sorted_rows(S, E, case["align"])
        return {"bytes": S * K + 4 * S * _blocks(K) + used * N * K + R * N * b,
                "flops": 2 * S * N * K}
    if op == "wgrad":
        S, E, M, N = (case[n] for n in ("S", "E", "M", "N"))
        return {"bytes": (S + S // 32) * (M + N) + E * M * N * DTYPES[case["out"]].itemsize,
                "flops": 2 * S * M * N}
    T, C, F, E, k = (case[n] for n in ("T", "C", "F", "E", "k"))
    b = DTYPES[case["weights"]].itemsize
    used = E * (1 - (1 - k / E) ** T)
    return {"bytes": used * 3 * C * F * b + 2 * T * C * DTYPES[case["dtype"]].itemsize + 8 * T * k,
            "flops": 6 * T * k * C * F}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_scales(v, fmt, dims):
    """v [B, 128, ...]: the largest magnitude over `dims` and the scale that goes with it."""
    a = torch.clamp_min(torch.amax(torch.abs(v), dims, keepdim=True), LEAST)
    return a, a / LARGEST[fmt]


def _exact_rows(v, fmt):
    """[R, C] float64 -> the quantised values and the scales [blocks, R], a block at a time."""
    q, s = torch.empty_like(v), v.new_empty(_blocks(v.shape[1]), v.shape[0])
    for j in range(s.shape[0]):
        part = v[:, j * BLOCK:(j + 1) * BLOCK]
        a, scale = _exact_scales(part, fmt, (1,))
        q[:, j * BLOCK:(j + 1) * BLOCK] = (part * (LARGEST[fmt] / a)).to(DTYPES[fmt]).double()
        s[j] = scale[:, 0]
    return q, s


def _exact_quant(v, mode, fmt):
    if mode == "tiles":
        R, C = v.shape
        q, s = torch.empty_like(v), v.new_empty(_blocks(C), _blocks(R))
        for i in range(s.shape[1]):
            rows = slice(i * BLOCK, (i + 1) * BLOCK)
            for j in range(s.shape[0]):
                cols = slice(j * BLOCK, (j + 1) * BLOCK)
                a, scale = _exact_scales(v[rows, cols], fmt, (0, 1))
                q[rows, cols] = (v[rows, cols] * (LARGEST[fmt] / a)).to(DTYPES[fmt]).double()
                s[j, i] = scale[0, 0]
        return {"q": q, "s": s, "qt": q.t().contiguous(), "st": s.t().contiguous()}
    out = {}
    if mode != "columns":
        out["q"], out["s"] = _exact_rows(v, fmt)
    if mode != "rows":
        out["qt"], out["st"] = _exact_rows(v.t().contiguous(), fmt)
    return out


def _exact_values(q, s):
    """[N, K] in 8 bits with scales [blocks of K, N or blocks of N] as float64."""
    v = q.double()
    for j in range(s.shape[0]):
        scale = s[j].double()
        if s.shape[1] != q.shape[0]:
            scale = scale[torch.arange(q.shape[0], device=q.device) // BLOCK]
        v[:, j * BLOCK:(j + 1) * BLOCK] *= scale[:, None]
    return v


def exact(case, seed):
    op = case["op"]
    if op in ("quant", "swiglu") and case["R"] * case.get("C", 2 * case.get("F", 0)) * case.get(
            "G", 1) > 700_000_000:
        return None
    s, f64 = prepare(case, seed), torch.float64
    if op == "quant":
        if case["G"] == 1:
            return _exact_quant(s["x"].to(f64), case["mode"], case["fmt"])
        each = [_exact_quant(x.to(f64), case["mode"], case["fmt"]) for x in s["x"]]
        return {n: torch.stack([e[n] for e in each]) for n in each[0]}
    if op == "swiglu":
        F, h = case["F"], s["h"].to(f64)
        gate, up = h[:, :F], h[:, F:]
        p = torch.sigmoid(gate)
        if case["way"] == "fwd":
            return _exact_quant(gate * p * up, case["mode"], case["fmt"])
        da = s["da"].to(f64)
        dh = torch.cat((da * up * (p + gate * p * torch.sigmoid(-gate)), da * gate * p), 1)
        return _exact_quant(dh, case["mode"], case["fmt"])
    if op in ("gemm", "wgrad"):
        at = s["offsets"].tolist()
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            if lo == hi:
                continue
            if op == "gemm":
                a = _exact_values(s["a"][lo:hi], s["sa"][:, lo:hi])
                out[lo:hi] = a @ _exact_values(s["b"][e], s["sb"][e]).t()
            else:
                rows = slice(lo // BLOCK, hi // BLOCK)
                a = _exact_values(s["at"][:, lo:hi], s["sat"][rows])
                out[e] = a @ _exact_values(s["bt"][:, lo:hi], s["sbt"][rows]).t()
        return {"out": out}
    x, ids, w = s["x"].to(f64), s["ids"], s["w"].to(f64)
    eight = s["s1"] is not None

    def as_quantised(v):
        if not eight:
            return v
        q, scale = _exact_rows(v, "e4m3")
        return _exact_values(q, scale)

    def weights(name, scales, e):
        return _exact_values(s[name][e], s[scales][e]) if eight else s[name][e].to(f64)

    x, f = as_quantised(x), torch.zeros_like(x)
    for e in sorted(set(ids.reshape(-1).tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = x[t] @ weights("w1", "s1", e).t()
        gate, up = h[:, :case["F"]], h[:, case["F"]:]
        a = as_quantised(gate * torch.sigmoid(gate) * up)
        f.index_add_(0, t, w[t, j][:, None] * (a @ weights("w2", "s2", e).t()))
    return {"f": f}
