"""The attention-entry and mixture-of-experts operators, as they are measured.

Five operators around the sub-layers that the residual path wraps: the norm of
queries and keys per head with the position rotation (qk), the router's top-k
(router), the sort of token slots by expert (sort), and the rows' way to the
experts and back (dispatch, combine), each with its gradient.  `own` chooses
between the library's calls and the same mathematics in elementary torch
operations, in fp32 and rounded once.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    qk = {"op": "qk", "Hq": 32, "Hk": 8, "D": 128, "R": 128, "P": 32768, "interleaved": False,
          "dtype": "bf16"}
    return [
        # one new token of one sequence while serving: latency alone
        {"name": "qk_fwd_token", "way": "fwd", "T": 1, **qk},
        # the attention entry of a training step, q and k as views of the packed qkv product
        {"name": "qk_fwd_layer", "way": "fwd", "T": 16384, **qk},
        # a ragged batch, head size off the powers of two, a quarter of it rotated, fp16
        {"name": "qk_fwd_partial", "way": "fwd", "T": 2999, **qk, "Hq": 20, "Hk": 20, "D": 80,
         "R": 20, "dtype": "fp16"},
        # the gradient of the training step's attention entry
        {"name": "qk_bwd_layer", "way": "bwd", "T": 16384, **qk},
        # the router of a training step over many experts, fp32 logits
        {"name": "router_fwd_layer", "op": "router", "way": "fwd", "T": 16384, "E": 256, "k": 8,
         "score": "softmax", "renorm": True, "scale": 1.0, "dtype": "fp32"},
        # its gradient, with sigmoid scores, bf16 logits and an odd number of experts
        {"name": "router_bwd_sigmoid", "op": "router", "way": "bwd", "T": 8192, "E": 61, "k": 4,
         "score": "sigmoid", "renorm": True, "scale": 2.5, "dtype": "bf16"},
        # the slots of a small serving batch
        {"name": "sort_batch", "op": "sort", "way": "fwd", "T": 37, "k": 4, "E": 60, "align": 16},
        # the slots of a training step, segments in tiles of a grouped product
        {"name": "sort_layer", "op": "sort", "way": "fwd", "T": 16384, "k": 8, "E": 256,
         "align": 128},
        # the rows of a training step to their experts
        {"name": "dispatch_fwd_layer", "op": "dispatch", "way": "fwd", "T": 16384, "C": 4096,
         "k": 4, "E": 64, "align": 128, "dtype": "bf16"},
        # the gradient of an odd, small batch in fp32
        {"name": "dispatch_bwd_ragged", "op": "dispatch", "way": "bwd", "T": 1001, "C": 7168,
         "k": 6, "E": 61, "align": 8, "dtype": "fp32"},
        # the experts' rows of a serving batch back to their tokens
        {"name": "combine_fwd_batch", "op": "combine", "way": "fwd", "T": 64, "C": 7168, "k": 8,
         "E": 256, "align": 8, "dtype": "bf16"},
        # the gradient of the way back, the wide model's training step
        {"name": "combine_bwd_wide", "op": "combine", "way": "bwd", "T": 8192, "C": 7168, "k": 8,
         "E": 256, "align": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk", "router", "sort", "dispatch", "combine"])
    way = "fwd" if op == "sort" else rng.choice(["fwd", "bwd"])
    T = _log_int(rng, 1, 16384)
    if op == "qk":
        D = rng.choice([64, 72, 80, 96, 112, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "way": way, "T": T, "Hq": Hk * rng.choice([1, 2, 4, 7]), "Hk": Hk,
                "D": D, "R": rng.choice([D, D, D // 2, 2 * (D // 8)]),
                "P": _log_int(rng, 16384, 131072), "interleaved": rng.random() < 0.3,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    E, k = _log_int(rng, 4, 512), rng.randint(1, 8)
    k = min(k, E)
    if op == "router":
        return {"op": op, "way": way, "T": T, "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    align = rng.choice([1, 8, 16, 128])
    if op == "sort":
        return {"op": op, "way": way, "T": T, "k": k, "E": E, "align": align}
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    C = 8 * _log_int(rng, 16, 896)
    most = (1 << 28) // (2 if dtype == "fp32" else 1)  # values of the sorted rows
    while T > 1 and _rows(T, k, E, align) * C > most:
        T = (T + 1) // 2
    if _rows(T, k, E, align) * C > most:
        align = 1
    return {"op": op, "way": way, "T": T, "C": C, "k": k, "E": E, "align": align, "dtype": dtype}


def _rows(T, k, E, align):
    """Rows that the sorted slots can take: every expert that has a slot pads its last tile."""
    return T * k + min(E, T * k) * (align - 1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ids(g, T, k, E):
    """Distinct experts per token, some experts far more popular; one slot in 64 is dropped."""
    popular = torch.log(torch.rand(E, generator=g, device="cuda") + 0.05)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda") * 0.9998 + 1e-4))
    ids = torch.topk(popular + noise, k, dim=1).indices.int()
    gone = torch.rand(T, k, generator=g, device="cuda") < 1 / 64
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    op, T = case["op"], case["T"]
    if op == "qk":
        Hq, Hk, D, R, P = (case[n] for n in ("Hq", "Hk", "D", "R", "P"))
        dt = DTYPES[case["dtype"]]
        qkv = _randn(g, T, Hq + 2 * Hk, D)
        qkv *= 0.25 + 2 * torch.rand(T, 1, 1, generator=g, device="cuda")
        qkv = qkv.to(dt)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["gamma_q"] = 1 + 0.1 * _randn(g, D)
        s["gamma_k"] = 1 + 0.1 * _randn(g, D)
        # the model's angle table, and sequences packed one after the other from any position
        inv = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2 / R)
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        docs = 1 + T // 1500
        start = torch.randint(0, P - T + 1, (docs,), generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["pos"] = (start[t * docs // T] + t % (1 + T // docs)).int().clamp_(0, P - 1)
        if case["way"] == "fwd":
            s["q_out"], s["k_out"] = _empty(T, Hq, D, dtype=dt), _empty(T, Hk, D, dtype=dt)
        else:
            s["dq_out"] = _randn(g, T, Hq, D).to(dt)
            s["dk_out"] = _randn(g, T, Hk, D).to(dt)
            s["dq"], s["dk"] = _empty(T, Hq, D, dtype=dt), _empty(T, Hk, D, dtype=dt)
            s["dgamma_q"], s["dgamma_k"] = _empty(D), _empty(D)
        return s
    if op == "router":
        E, k, dt = case["E"], case["k"], DTYPES[case["dtype"]]
        s["logits"] = (1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)).to(dt)
        s["ids"], s["w"] = _empty(T, k, dtype=torch.int32), _empty(T, k)
        if case["way"] == "bwd":
            s["ids"].copy_(_choose(s["logits"], k))
            s["dw"], s["dlogits"] = _randn(g, T, k), _empty(T, E, dtype=dt)
        return s
    E, k, align = case["E"], case["k"], case["align"]
    rows = _rows(T, k, E, align)
    s["ids"] = _ids(g, T, k, E)
    if op == "sort":
        i32 = torch.int32
        s["counts"], s["offsets"] = _empty(E, dtype=i32), _empty(E + 1, dtype=i32)
        s["row_of"], s["slot_of"] = _empty(T, k, dtype=i32), _empty(rows, dtype=i32)
        return s
    _, _, s["row_of"], s["slot_of"] = _plan(s["ids"], E, align, rows)
    C, dt = case["C"], DTYPES[case["dtype"]]
    if op == "dispatch" and case["way"] == "fwd":
        s["x"], s["xs"] = _randn(g, T, C).to(dt), _empty(rows, C, dtype=dt)
    elif op == "dispatch":
        s["dxs"], s["dx"] = _randn(g, rows, C).to(dt), _empty(T, C, dtype=dt)
    else:
        s["ys"] = _randn(g, rows, C).to(dt)
        w = torch.rand(T, k, generator=g, device="cuda") + 0.02
        s["w"] = w / w.sum(1, keepdim=True)
        if case["way"] == "fwd":
            s["f"] = _empty(T, C, dtype=dt)
        else:
            s["df"] = _randn(g, T, C).to(dt)
            s["dys"], s["dw"] = _empty(rows, C, dtype=dt), _empty(T, k)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _halves(x, R, interleaved):
    if interleaved:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _joined(a, b, rest, interleaved):
    ab = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _plain_qk_fwd(x, gamma, cos, sin, R, interleaved):
    xf = x.float()
    a = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6) * gamma
    u, v = _halves(a, R, interleaved)
    return _joined(u * cos - v * sin, v * cos + u * sin, a[..., R:], interleaved).to(x.dtype)


def _plain_qk_bwd(dy, x, gamma, cos, sin, R, interleaved):
    xf, dyf = x.float(), dy.float()
    rho = torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6)
    u, v = _halves(dyf, R, interleaved)
    b = _joined(u * cos + v * sin, v * cos - u * sin, dyf[..., R:], interleaved)
    xh, g = xf * rho, b * gamma
    dx = rho * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (b * xh).sum((0, 1))


def _choose(logits, k):
    """The k largest logits of each row, ties to the lowest index."""
    return torch.sort(logits.float(), dim=-1, descending=True, stable=True).indices[:, :k].int()


def _plain_router_fwd(logits, k, score, renorm, scale):
    ids = _choose(logits, k)
    lf = logits.float()
    at = ids.long()
    if score == "softmax":
        p = torch.exp(lf - lf.amax(-1, keepdim=True))
    else:
        p = 1 / (1 + torch.exp(-lf))
    c = p.gather(1, at)
    if renorm:
        c = c / c.sum(-1, keepdim=True)
    elif score == "softmax":
        c = c / p.sum(-1, keepdim=True)
    return ids, scale * c


def _plain_router_bwd(dw, logits, ids, score, renorm, scale):
    lf, at, a = logits.float(), ids.long(), scale * dw
    if score == "softmax":
        p = torch.exp(lf - lf.amax(-1, keepdim=True))
    else:
        p = 1 / (1 + torch.exp(-lf))
    c = p.gather(1, at)
    if score == "softmax" and not renorm:
        p = p / p.sum(-1, keepdim=True)
        inner = (a * p.gather(1, at)).sum(-1, keepdim=True)
        return (p * (torch.zeros_like(lf).scatter(1, at, a) - inner)).to(logits.dtype)
    if renorm:
        w = c / c.sum(-1, keepdim=True)
        d = w * (a - (a * w).sum(-1, keepdim=True))
        if score == "sigmoid":
            d = d * (1 - c)
    else:
        d = a * c * (1 - c)
    return torch.zeros_like(lf).scatter(1, at, d).to(logits.dtype)


def _plan(ids, E, align, rows):
    """counts, offsets, row_of, slot_of of a stable sort by expert, in tiles of `align` rows."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    first = counts.cumsum(0) - counts
    tiles = (counts[:E] + align - 1) // align * align
    offsets = torch.cat((torch.zeros_like(counts[:1]), tiles.cumsum(0)))
    kept = key < E
    dest = offsets[key] + torch.arange(T * k, device=ids.device) - first[key]
    row_of = torch.empty_like(flat)
    row_of.scatter_(0, order, torch.where(kept, dest, torch.full_like(dest, -1)))
    slot_of = torch.full((rows + 1,), -1, dtype=torch.int64, device=ids.device)
    slot_of.scatter_(0, torch.where(kept, dest, torch.full_like(dest, rows)), order)
    return (counts[:E].int(), offsets.int(), row_of.int().reshape(T, k),
            slot_of[:rows].int().contiguous())


def _by_slot(per_token, slot_of, k):
    """Row r of the sorted order holds its slot's token row, 0 where it has no slot."""
    slot = slot_of.long()
    rows = per_token[slot.clamp(min=0) // k]
    return torch.where((slot >= 0)[:, None], rows, torch.zeros_like(rows))


def _by_token(rows, row_of):
    """[T, k, C]: the sorted rows of each token's slots, 0 for a dropped slot."""
    at = row_of.long()
    got = rows[at.clamp(min=0)]
    return torch.where((at >= 0)[..., None], got, torch.zeros_like(got))


def _plain(s):
    c = s["case"]
    op, way = c["op"], c["way"]
    if op == "qk":
        at = s["pos"].long()
        rope = (s["cos"][at][:, None], s["sin"][at][:, None], c["R"], c["interleaved"])
        if way == "fwd":
            return {"q": _plain_qk_fwd(s["q"], s["gamma_q"], *rope),
                    "k": _plain_qk_fwd(s["k"], s["gamma_k"], *rope)}
        dq, dgq = _plain_qk_bwd(s["dq_out"], s["q"], s["gamma_q"], *rope)
        dk, dgk = _plain_qk_bwd(s["dk_out"], s["k"], s["gamma_k"], *rope)
        return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}
    if op == "router":
        how = (c["score"], c["renorm"], c["scale"])
        if way == "fwd":
            ids, w = _plain_router_fwd(s["logits"], c["k"], *how)
            return {"ids": ids, "w": w}
        return {"dlogits": _plain_router_bwd(s["dw"], s["logits"], s["ids"], *how)}
    if op == "sort":
        rows = s["slot_of"].shape[0]
        return dict(zip(("counts", "offsets", "row_of", "slot_of"),
                        _plan(s["ids"], c["E"], c["align"], rows)))
    if op == "dispatch" and way == "fwd":
        return {"xs": _by_slot(s["x"], s["slot_of"], c["k"])}
    if op == "dispatch":
        return {"dx": _by_token(s["dxs"], s["row_of"]).float().sum(1).to(s["dxs"].dtype)}
    got = _by_token(s["ys"], s["row_of"]).float()
    if way == "fwd":
        return {"f": (s["w"][..., None] * got).sum(1).to(s["ys"].dtype)}
    dff = s["df"].float()
    weight = s["w"].reshape(-1)[s["slot_of"].long().clamp(min=0)]
    return {"dys": (weight[:, None] * _by_slot(dff, s["slot_of"], c["k"])).to(s["ys"].dtype),
            "dw": (got * dff[:, None]).sum(-1)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import layers_proj_rms_gb300 as M
    c = s["case"]
    op, way = c["op"], c["way"]
    if op == "qk" and way == "fwd":
        M.mhc_qk_norm_rope_fwd(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["cos"], s["sin"],
                               s["pos"], 1e-6, s["q_out"], s["k_out"],
                               interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "qk":
        if "ws" not in s:
            s["ws"] = M.workspace(M.OP_QK_NORM_ROPE_BWD, c["T"], c["Hq"] + c["Hk"], c["D"])
        M.mhc_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["gamma_q"],
                               s["gamma_k"], s["cos"], s["sin"], s["pos"], 1e-6, s["dq"], s["dk"],
                               s["dgamma_q"], s["dgamma_k"], s["ws"],
                               interleaved=c["interleaved"])
        return {n: s[n] for n in ("dq", "dk", "dgamma_q", "dgamma_k")}
    if op == "router":
        score = M.SCORE_SOFTMAX if c["score"] == "softmax" else M.SCORE_SIGMOID
        if way == "fwd":
            M.mhc_moe_router_fwd(s["logits"], score, c["renorm"], c["scale"], s["ids"], s["w"])
            return {"ids": s["ids"], "w": s["w"]}
        M.mhc_moe_router_bwd(s["dw"], s["logits"], s["ids"], score, c["renorm"], c["scale"],
                             s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "sort":
        M.mhc_moe_sort(s["ids"], c["align"], s["counts"], s["offsets"], s["row_of"], s["slot_of"])
        return {n: s[n] for n in ("counts", "offsets", "row_of", "slot_of")}
    if op == "dispatch" and way == "fwd":
        M.mhc_moe_dispatch_fwd(s["x"], s["row_of"], s["slot_of"], s["xs"])
        return {"xs": s["xs"]}
    if op == "dispatch":
        M.mhc_moe_dispatch_bwd(s["dxs"], s["row_of"], s["dx"])
        return {"dx": s["dx"]}
    if way == "fwd":
        M.mhc_moe_combine_fwd(s["ys"], s["w"], s["row_of"], s["f"])
        return {"f": s["f"]}
    M.mhc_moe_combine_bwd(s["df"], s["ys"], s["w"], s["row_of"], s["slot_of"], s["dys"], s["dw"])
    return {"dys": s["dys"], "dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, way, T = case["op"], case["way"], case["T"]
    if op == "qk":
        b = DTYPES[case["dtype"]].itemsize
        n = T * (case["Hq"] + case["Hk"]) * case["D"]
        table = T * 4 + min(T, case["P"]) * case["R"] * 4 + case["D"] * 8
        if way == "fwd":
            return {"bytes": 2 * n * b + table, "flops": 8 * n}
        return {"bytes": 3 * n * b + table + case["D"] * 8, "flops": 18 * n}
    if op == "router":
        n, b, k = T * case["E"], DTYPES[case["dtype"]].itemsize, case["k"]
        if way == "fwd":
            return {"bytes": n * b + T * k * 8, "flops": 4 * n}
        return {"bytes": 2 * n * b + T * k * 8, "flops": 6 * n}
    k, E = case["k"], case["E"]
    rows = _rows(T, k, E, case["align"])
    if op == "sort":
        return {"bytes": 4 * (2 * T * k + rows + 2 * E + 1), "flops": 4 * T * k}
    b, C = DTYPES[case["dtype"]].itemsize, case["C"]
    if op == "dispatch" and way == "fwd":
        return {"bytes": (T + rows) * C * b + 4 * (T * k + rows), "flops": 0}
    if op == "dispatch":
        return {"bytes": (T + T * k) * C * b + 4 * T * k, "flops": T * k * C}
    if way == "fwd":
        return {"bytes": (T + T * k) * C * b + 8 * T * k, "flops": 2 * T * k * C}
    return {"bytes": (T + T * k + rows) * C * b + 4 * (3 * T * k + rows), "flops": 3 * T * k * C}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_qk(s, c, x, gamma, dy=None):
    f64 = torch.float64
    x, gamma = x.to(f64), gamma.to(f64)
    D, h = x.shape[-1], c["R"] // 2
    j = torch.arange(D, device=x.device)
    rotated = j < 2 * h
    if c["interleaved"]:
        pair, first, partner = j // 2, j % 2 == 0, j ^ 1
    else:
        pair, first = j % max(h, 1), j < h
        partner = torch.where(first, j + h, j - h)
    partner = torch.where(rotated, partner, j)
    pair = torch.where(rotated, pair, torch.zeros_like(j))
    at = s["pos"].long()
    cos = torch.where(rotated, s["cos"][at].to(f64)[:, pair], 1.0)[:, None]
    sin = torch.where(rotated, s["sin"][at].to(f64)[:, pair], 0.0)[:, None]
    sin = torch.where(first, -sin, sin)
    norm = ((x * x).sum(-1, keepdim=True) / D + 1e-6).sqrt()
    if dy is None:
        a = x / norm * gamma
        return a * cos + a[..., partner] * sin
    dy = dy.to(f64)
    b = dy * cos - dy[..., partner] * sin
    u = x / norm
    inner = (b * gamma * u).sum(-1, keepdim=True) / D
    return (b * gamma - u * inner) / norm, (b * u).sum(1).sum(0)


def exact(case, seed):
    op, way = case["op"], case["way"]
    if op == "sort":
        return None
    s, f64 = prepare(case, seed), torch.float64
    if op == "qk" and way == "fwd":
        return {"q": _exact_qk(s, case, s["q"], s["gamma_q"]),
                "k": _exact_qk(s, case, s["k"], s["gamma_k"])}
    if op == "qk":
        dq, dgq = _exact_qk(s, case, s["q"], s["gamma_q"], s["dq_out"])
        dk, dgk = _exact_qk(s, case, s["k"], s["gamma_k"], s["dk_out"])
        return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}
    if op == "router":
        l = s["logits"].to(f64)
        ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        if way == "bwd":
            ids = s["ids"].long()
        chosen = torch.zeros_like(l, dtype=torch.bool).scatter(1, ids, True)
        score = -torch.log1p(torch.exp(-l)) if case["score"] == "sigmoid" else l
        over = chosen if case["renorm"] else torch.ones_like(chosen)
        if case["score"] == "sigmoid" and not case["renorm"]:
            p = torch.sigmoid(l)
        else:
            p = torch.softmax(torch.where(over, score, -math.inf), dim=1)
        if way == "fwd":
            return {"ids": None, "w": case["scale"] * p.gather(1, ids)}
        up = torch.zeros_like(l).scatter(1, ids, case["scale"] * s["dw"].to(f64))
        slope = torch.sigmoid(-l) if case["score"] == "sigmoid" else torch.ones_like(l)
        if case["score"] == "sigmoid" and not case["renorm"]:
            return {"dlogits": up * p * slope}
        return {"dlogits": p * slope * (up - (p * up).sum(1, keepdim=True))}
    k, row, slot = case["k"], s["row_of"].long(), s["slot_of"].long()
    T, C = case["T"], case["C"]
    if op == "dispatch" and way == "fwd":
        xs = torch.zeros(slot.shape[0], C, dtype=f64, device=slot.device)
        held = slot >= 0
        xs[held] = s["x"].to(f64)[slot[held] // k]
        return {"xs": xs}
    kept = (row >= 0).reshape(-1)
    token = torch.arange(T, device=row.device).repeat_interleave(k)[kept]
    row = row.reshape(-1)[kept]
    if op == "dispatch":
        dx = torch.zeros(T, C, dtype=f64, device=row.device)
        return {"dx": dx.index_add_(0, token, s["dxs"][row].to(f64))}
    w = s["w"].to(f64).reshape(-1)[kept]
    if way == "fwd":
        f = torch.zeros(T, C, dtype=f64, device=row.device)
        return {"f": f.index_add_(0, token, w[:, None] * s["ys"][row].to(f64))}
    dys = torch.zeros(slot.shape[0], C, dtype=f64, device=row.device)
    dys[row] = w[:, None] * s["df"].to(f64)[token]
    dw = torch.zeros(T * k, dtype=f64, device=row.device)
    part = [(s["ys"][r].to(f64) * s["df"].to(f64)[t]).sum(1)
            for r, t in zip(row.split(1 << 14), token.split(1 << 14))]
    dw[kept] = torch.cat(part) if part else dw[:0]
    return {"dys": dys, "dw": dw.reshape(T, k)}
