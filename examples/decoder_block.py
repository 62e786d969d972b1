"""One decoder block on the n-stream residual, forward and backward: an mHC
layer around attention and one around a mixture of experts.

    x [T, n, C] -> controller (H_pre, H_post, H_res) -> y = RMSNorm(aggregate)
    attention:  qkv = y Wqkv -> q/k norm + rotation -> causal attention -> Wo
    experts:    router -> sort -> dispatch -> expert products -> combine
    -> post-mix with the residual, once per layer

The steps around the matrix products are libmhc's; the products themselves and
the attention core are torch's.  `python examples/decoder_block.py` runs a step
and compares its gradients with torch's autograd on the same block.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layers_proj_rms_gb300 as M  # noqa: E402

EPS, ITERS = 1e-6, 20
BF, F32 = torch.bfloat16, torch.float32


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def make(T=256, n=4, C=512, Hq=8, Hk=2, D=64, E=8, k=2, F=256, align=16, seed=0):
    """Sizes, weights, an input and an upstream gradient."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0, dtype=BF: (std * torch.randn(*s, generator=g, device="cuda")).to(dtype)  # noqa: E731
    O = n * n + 2 * n
    layer = lambda: {"W": rnd(n * C, O, std=0.02, dtype=F32), "b": rnd(O, std=0.5, dtype=F32),  # noqa: E731
                     "alpha": torch.full((3,), 0.5, device="cuda"), "bias": rnd(C, std=0.02),
                     "gamma": 1 + rnd(C, std=0.1, dtype=F32)}
    angle = torch.arange(T, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(D // 2, device="cuda") * 2.0 / D)
    p = {"attn": {**layer(), "Wqkv": rnd(C, (Hq + 2 * Hk) * D, std=C ** -0.5),
                  "Wo": rnd(Hq * D, C, std=(Hq * D) ** -0.5),
                  "gamma_q": 1 + rnd(D, std=0.1, dtype=F32), "gamma_k": 1 + rnd(D, std=0.1, dtype=F32)},
         "moe": {**layer(), "Wr": rnd(C, E, std=C ** -0.5, dtype=F32),
                 "W1": rnd(E, C, F, std=C ** -0.5), "W2": rnd(E, F, C, std=F ** -0.5)},
         "cos": angle.cos(), "sin": angle.sin(),
         "pos": torch.arange(T, dtype=torch.int32, device="cuda")}
    size = {"T": T, "n": n, "C": C, "Hq": Hq, "Hk": Hk, "D": D, "E": E, "k": k, "align": align}
    return size, p, rnd(T, n, C), rnd(T, n, C)


# ---- what both layers share: into the sub-layer, and back into the residual ----

def enter(s, w, x):
    """H_*, and the normalised aggregate that the sub-layer reads."""
    T, n, C = x.shape
    O = n * n + 2 * n
    c = {"x": x, "H_pre": empty(T, n, dtype=F32), "H_post": empty(T, n, dtype=F32),
         "H_res": empty(T, n, n, dtype=F32), "u": empty(T, O, dtype=F32), "r": empty(T, dtype=F32),
         "y": empty(T, C), "yn": empty(T, C), "rstd": empty(T, dtype=F32)}
    M.mhc_proj_rms_compute_h_fwd(x, w["W"], w["alpha"], w["b"], ITERS, EPS, EPS, c["H_pre"],
                                 c["H_post"], c["H_res"], c["u"], c["r"],
                                 M.workspace(M.OP_PROJ_RMS_COMPUTE_H_FWD, T, n, C))
    M.mhc_h_aggregate_rmsnorm_fwd(x, c["H_pre"], w["gamma"], c["y"], c["yn"], c["rstd"], EPS)
    return c


def leave(w, c, f):
    c["f"], out = f, torch.empty_like(c["x"])
    M.mhc_h_post_bda_fwd(c["x"], f, w["bias"], c["H_res"], c["H_post"], out)
    return out


def leave_bwd(w, c, dout, grads):
    """df; keeps the gradients of the residual and of H_post, H_res."""
    T, n, C = dout.shape
    c["dres"], df = torch.empty_like(dout), empty(T, C)
    grads["bias"] = empty(C, dtype=F32)
    c["dH_res"], c["dH_post"] = torch.empty_like(c["H_res"]), torch.empty_like(c["H_post"])
    M.mhc_h_post_bda_bwd(dout, c["x"], c["f"], w["bias"], c["H_res"], c["H_post"], c["dres"], df,
                         grads["bias"], c["dH_res"], c["dH_post"],
                         M.workspace(M.OP_H_POST_BDA_BWD, T, n, C))
    return df


def enter_bwd(w, c, dyn, grads):
    """dx of the layer from the gradient of the normalised aggregate."""
    x = c["x"]
    T, n, C = x.shape
    dx_agg, dx_proj = torch.empty_like(x), torch.empty_like(x)
    dH_pre = torch.empty_like(c["H_pre"])
    for name in ("W", "b", "alpha", "gamma"):
        grads[name] = torch.empty_like(w[name])
    M.mhc_h_aggregate_rmsnorm_bwd(dyn, None, x, c["H_pre"], w["gamma"], c["rstd"], dx_agg, dH_pre,
                                  grads["gamma"], EPS,
                                  M.workspace(M.OP_H_AGGREGATE_RMSNORM_BWD, T, n, C))
    M.mhc_proj_rms_compute_h_bwd(dH_pre, c["dH_post"], c["dH_res"], x, w["W"], w["alpha"], w["b"],
                                 c["u"], c["r"], ITERS, EPS, EPS, dx_proj, grads["W"],
                                 grads["alpha"], grads["b"],
                                 M.workspace(M.OP_PROJ_RMS_COMPUTE_H_BWD, T, n, C))
    return (c["dres"].float() + dx_agg.float() + dx_proj.float()).to(BF)


# ---- attention -----------------------------------------------------------------

def attend(q, k, v):
    """Causal attention over heads in groups: [T, H, D] each."""
    T, Hq, D = q.shape
    k, v = (t.repeat_interleave(Hq // t.shape[1], 1) for t in (k, v))
    a = torch.einsum("qhd,khd->hqk", q.float(), k.float()) * D ** -0.5
    a = a.masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return torch.einsum("hqk,khd->qhd", a.softmax(-1), v.float())


def attention(s, p, w, yn):
    T, Hq, Hk, D = s["T"], s["Hq"], s["Hk"], s["D"]
    qkv = (yn @ w["Wqkv"]).view(T, Hq + 2 * Hk, D)
    q, k, v = qkv.split((Hq, Hk, Hk), 1)  # views of the packed product
    qr, kr = empty(T, Hq, D), empty(T, Hk, D)
    M.mhc_qk_norm_rope_fwd(q, k, w["gamma_q"], w["gamma_k"], p["cos"], p["sin"], p["pos"], EPS, qr, kr)
    leaf = [t.detach().requires_grad_() for t in (qr, kr, v)]
    with torch.enable_grad():
        o = attend(*leaf).to(BF)
    return o.detach().flatten(1) @ w["Wo"], {"yn": yn, "q": q, "k": k, "leaf": leaf, "o": o}


def attention_bwd(s, p, w, c, df, grads):
    T, Hq, Hk, D = s["T"], s["Hq"], s["Hk"], s["D"]
    grads["Wo"] = c["o"].detach().flatten(1).T @ df
    dqr, dkr, dv = torch.autograd.grad(c["o"], c["leaf"], (df @ w["Wo"].T).view(T, Hq, D))
    dqkv = empty(T, Hq + 2 * Hk, D)
    dq, dk, dv_ = dqkv.split((Hq, Hk, Hk), 1)  # the gradients go into the packed product's
    dv_.copy_(dv)
    grads["gamma_q"], grads["gamma_k"] = torch.empty_like(w["gamma_q"]), torch.empty_like(w["gamma_k"])
    M.mhc_qk_norm_rope_bwd(dqr, dkr, c["q"], c["k"], w["gamma_q"], w["gamma_k"], p["cos"], p["sin"],
                           p["pos"], EPS, dq, dk, grads["gamma_q"], grads["gamma_k"],
                           M.workspace(M.OP_QK_NORM_ROPE_BWD, T, Hq + Hk, D))
    dqkv = dqkv.flatten(1)
    grads["Wqkv"] = c["yn"].T @ dqkv
    return dqkv @ w["Wqkv"].T


# ---- mixture of experts ----------------------------------------------------------

def experts(s, p, w, yn):
    T, C, E, k, align = s["T"], s["C"], s["E"], s["k"], s["align"]
    R = M.mhc_moe_rows(T, k, E, align)
    i32 = torch.int32
    c = {"yn": yn, "logits": yn.float() @ w["Wr"], "ids": empty(T, k, dtype=i32),
         "w": empty(T, k, dtype=F32), "row_of": empty(T, k, dtype=i32), "slot_of": empty(R, dtype=i32),
         "xs": empty(R, C), "ys": torch.zeros(R, C, dtype=BF, device="cuda")}
    counts, offsets = empty(E, dtype=i32), empty(E + 1, dtype=i32)
    M.mhc_moe_router_fwd(c["logits"], M.SCORE_SOFTMAX, True, 1.0, c["ids"], c["w"])
    M.mhc_moe_sort(c["ids"], align, counts, offsets, c["row_of"], c["slot_of"])
    M.mhc_moe_dispatch_fwd(yn, c["row_of"], c["slot_of"], c["xs"])
    # a grouped product would read the offsets on the device
    c["seg"] = offsets.tolist()
    c["h"] = [c["xs"][a:b] @ w["W1"][e] for e, (a, b) in enumerate(zip(c["seg"], c["seg"][1:]))]
    for e, (a, b) in enumerate(zip(c["seg"], c["seg"][1:])):
        c["ys"][a:b] = torch.relu(c["h"][e]) @ w["W2"][e]
    f = empty(T, C)
    M.mhc_moe_combine_fwd(c["ys"], c["w"], c["row_of"], f)
    return f, c


def experts_bwd(s, p, w, c, df, grads):
    dys, dxs = torch.empty_like(c["ys"]), torch.zeros_like(c["xs"])
    dw, dl, dx = torch.empty_like(c["w"]), torch.empty_like(c["logits"]), torch.empty_like(c["yn"])
    M.mhc_moe_combine_bwd(df, c["ys"], c["w"], c["row_of"], c["slot_of"], dys, dw)
    grads["W1"], grads["W2"] = torch.empty_like(w["W1"]), torch.empty_like(w["W2"])
    for e, (a, b) in enumerate(zip(c["seg"], c["seg"][1:])):
        h, d = c["h"][e], dys[a:b]
        grads["W2"][e] = torch.relu(h).T @ d
        dh = (d @ w["W2"][e].T) * (h > 0)
        grads["W1"][e] = c["xs"][a:b].T @ dh
        dxs[a:b] = dh @ w["W1"][e].T
    M.mhc_moe_dispatch_bwd(dxs, c["row_of"], dx)
    M.mhc_moe_router_bwd(dw, c["logits"], c["ids"], M.SCORE_SOFTMAX, True, 1.0, dl)
    grads["Wr"] = c["yn"].float().T @ dl
    return (dx.float() + dl @ w["Wr"].T).to(BF)


# ---- the block -------------------------------------------------------------------

def forward(s, p, x):
    caches = []
    for name, sub in (("attn", attention), ("moe", experts)):
        w = p[name]
        c = enter(s, w, x)
        f, inner = sub(s, p, w, c["yn"])
        x = leave(w, c, f)
        caches.append((c, inner))
    return x, caches


def backward(s, p, caches, dout):
    grads = {"attn": {}, "moe": {}}
    for name, sub, (c, inner) in (("moe", experts_bwd, caches[1]), ("attn", attention_bwd, caches[0])):
        w, g = p[name], grads[name]
        df = leave_bwd(w, c, dout, g)
        dout = enter_bwd(w, c, sub(s, p, w, inner, df, g), g)
    return dout, grads


# ---- the same block in plain torch, fp32, with autograd ----------------------------

def reference(s, p, x, ids, through=lambda path, v: v):
    """through(path, v) stands for v on one of the ways from x to the output (an
    identity, but for its gradient if a caller wants to cut one)."""
    def controller(w, x):
        T, n, C = x.shape
        flat = x.flatten(1)
        z = flat @ w["W"] / (flat.square().mean(-1, keepdim=True).sqrt() + EPS)
        a = torch.cat([w["alpha"][i].expand(m) for i, m in enumerate((n, n, n * n))])
        z = z * a + w["b"]
        P = z[:, 2 * n:].view(T, n, n).exp()
        for _ in range(ITERS):
            P = P / (P.sum(-1, keepdim=True) + EPS)
            P = P / (P.sum(-2, keepdim=True) + EPS)
        return z[:, :n].sigmoid(), 2 * z[:, n:2 * n].sigmoid(), P

    def norm(v, g):
        return v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * g

    def rope(v):
        a, b = v.chunk(2, -1)
        c, d = p["cos"][:, None], p["sin"][:, None]
        return torch.cat((a * c - b * d, b * c + a * d), -1)

    for name in ("attn", "moe"):
        w = p[name]
        at = lambda path, v: through(f"{name}.{path}", v)  # noqa: E731, B023
        pre, post, res = (at(n, h) for n, h in zip(("H_pre", "H_post", "H_res"), controller(w, x)))
        y = norm(torch.einsum("tn,tnc->tc", pre, at("aggregate", x)), w["gamma"])
        if name == "attn":
            q, k, v = (y @ w["Wqkv"]).view(s["T"], -1, s["D"]).split((s["Hq"], s["Hk"], s["Hk"]), 1)
            q, k, v = at("q", q), at("k", k), at("v", v)
            f = attend(rope(norm(q, w["gamma_q"])), rope(norm(k, w["gamma_k"])), v).flatten(1) @ w["Wo"]
        else:
            wt = (at("router", y) @ w["Wr"]).gather(1, ids.long()).softmax(-1)
            h = torch.einsum("tc,ecf->tef", at("experts", y), w["W1"]).relu()
            each = torch.einsum("tef,efc->tec", h, w["W2"])
            f = torch.einsum("tk,tkc->tc", wt, each.gather(
                1, ids.long()[..., None].expand(-1, -1, s["C"])))
        x = torch.einsum("tji,tjc->tic", res, at("residual", x)) + post[..., None] * (f + w["bias"])[:, None]
    return x


def compare(s, p, x, dout):
    """Relative errors of the output and every gradient against the reference."""
    out, caches = forward(s, p, x)
    dx, grads = backward(s, p, caches, dout)
    leaf = {a: {n: t.float().detach().requires_grad_() for n, t in p[a].items()} for a in ("attn", "moe")}
    xr = x.float().detach().requires_grad_()
    ref = reference(s, {**p, **leaf}, xr, caches[1][1]["ids"])
    names = [(a, n) for a in leaf for n in leaf[a]]
    want = torch.autograd.grad(ref, [xr] + [leaf[a][n] for a, n in names], dout.float())
    rel = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    errs = {"out": rel(out, ref.detach()), "dx": rel(dx, want[0])}
    errs.update({f"{a}.{n}": rel(grads[a][n], g) for (a, n), g in zip(names, want[1:])})
    return errs


if __name__ == "__main__":
    errors = compare(*make())
    for name, e in errors.items():
        print(f"{name:16s} relative error {e:.2e}")
    print("device error", M.mhc_device_error())
