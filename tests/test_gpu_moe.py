"""Router, sort, dispatch and combine on the GPU against the plain 64-bit forms
(tests/_edges.py says how the tolerances come about)."""
import numpy as np
import pytest
import torch

from tests import _edges as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def rng(seed):
    return torch.Generator().manual_seed(seed)


def i32(*s):
    return torch.full(s, 77, dtype=torch.int32, device="cuda")


def route(M, logits, k, score, renorm, scale=1.0):
    T = logits.shape[0]
    ids, w = i32(T, k), torch.full((T, k), 7.0, device="cuda")
    M.mhc_moe_router_fwd(logits, M.SCORE_SOFTMAX if score == "softmax" else M.SCORE_SIGMOID,
                         renorm, scale, ids, w)
    return ids, w


def route_bwd(M, dw, logits, ids, score, renorm, scale=1.0):
    out = torch.full_like(logits, 7)
    M.mhc_moe_router_bwd(dw, logits, ids, M.SCORE_SOFTMAX if score == "softmax" else
                         M.SCORE_SIGMOID, renorm, scale, out)
    return out


# exp is off by 2 steps and by the rounding of its argument times |argument|
def exp_ops(l, n):
    return n + 16 + 8 * np.abs(l[np.isfinite(l)]).max(initial=0.0)


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (37, 61, 4), (130, 8, 8), (9, 1024, 32),
                                   (64, 128, 1), (33, 384, 6), (5, 33, 32), (7, 512, 8)])
def test_router(M, T, E, k, score, renorm, dt):
    g = rng(T + E)
    l = (2 * torch.randn(T, E, generator=g)).to(dt).cuda()
    ids, w = route(M, l, k, score, renorm, 2.5)
    ln, idn = O.np64(l), ids.cpu().numpy()
    assert np.array_equal(idn, O.top(ln, k))
    ref = 2.5 * O.router_scores(ln, idn, score, renorm)
    O.check(w, ref, ref, exp_ops(ln, E), "w")
    dw = torch.randn(T, k, generator=g).cuda()
    if k > 1:
        ids[T // 2, k // 2] = -1  # a slot dropped after the choice
    got = route_bwd(M, dw, l, ids, score, renorm, 2.5)
    d, dm = O.router_bwd(O.np64(dw), ln, ids.cpu().numpy(), score, renorm, 2.5)
    O.check(got, d, dm, 2 * exp_ops(ln, E) + k, "dlogits")
    assert M.mhc_device_error() == 0


def test_router_ties_masks_and_nan(M):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    l = torch.tensor([[1.0, 1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -0.0, -1, 0],
                      [-inf, -inf, 3, -inf, 3, -inf], [-inf] * 6, [low] * 6,
                      [-inf, nan, 5, 1, nan, 0], [2, 90, -90, 100, 3, -200]], device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = route(M, l, 3, score, renorm)
            assert ids.tolist()[:5] == [[0, 1, 2], [0, 1, 2], [2, 4, 0], [0, 1, 2], [0, 1, 2]]
            assert ids.tolist()[5:] == [[1, 4, 2], [3, 1, 4]]
            assert torch.all(w[3] == 0) and w[2, 2] == 0
            assert w[2, 0] == w[2, 1] > 0 and torch.all(torch.isfinite(w[[0, 1, 2, 3, 4, 6]]))
            assert torch.isnan(w[5, 0])  # a NaN logit is not hidden
            if renorm:
                assert torch.allclose(w[4], torch.full((3,), 1 / 3, device="cuda"))
            d = route_bwd(M, torch.ones_like(w), l, ids, score, renorm)
            assert torch.all(torch.isfinite(d[[0, 1, 2, 3, 4, 6]])) and torch.all(d[3] == 0)
    # nothing chosen at all; an id that is no expert is left out and reported
    none = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    fine = l[:5].contiguous()
    d = route_bwd(M, torch.ones(5, 3, device="cuda"), fine, none, "softmax", True)
    assert torch.all(d == 0) and M.mhc_device_error() == 0
    none[0, 0] = 6
    route_bwd(M, torch.ones(5, 3, device="cuda"), fine, none, "softmax", True)
    assert M.mhc_device_error() == 204 and M.mhc_device_error() == 0


def test_router_bf16_ties_are_common_and_exact(M):
    l = (torch.randint(0, 6, (300, 256), generator=rng(3)).float() / 4).bfloat16().cuda()
    ids, _ = route(M, l, 8, "softmax", True)
    assert np.array_equal(ids.cpu().numpy(), O.top(O.np64(l), 8))


@pytest.mark.parametrize("E,k", [(64, 4), (200, 8), (256, 8), (1024, 32)])
def test_router_logits_that_differ_in_their_last_bits(M, E, k):
    """fp32 logits a few steps apart (all, or some at the border of the choice),
    and every kind of 16-bit pattern."""
    g = rng(E)
    near = torch.stack([torch.randperm(E, generator=g) for _ in range(40)]).int()
    base = torch.tensor([1.0, -1.0, 3e-39, 2.5e38]).view(torch.int32).repeat(10)[:, None]
    l = (base + near).view(torch.float32)
    l[10:20] = torch.where(near[10:20] % 3 == 0, l[10:20], torch.randn(10, E, generator=g))
    ids, w = route(M, l.cuda(), k, "softmax", True)
    assert np.array_equal(ids.cpu().numpy(), O.top(l.double().numpy(), k))
    for dt in (torch.bfloat16, torch.float16):
        bits = torch.randint(-32768, 32768, (200, E), generator=g).to(torch.int16).view(dt)
        bits = torch.where(bits.isfinite(), bits, torch.zeros((), dtype=dt))
        ids, _ = route(M, bits.cuda(), k, "sigmoid", False)
        assert np.array_equal(ids.cpu().numpy(), O.top(bits.double().numpy(), k))


def plan(M, ids, E, align, R=None):
    T, k = ids.shape
    R = M.mhc_moe_rows(T, k, E, align) if R is None else R
    out = i32(E), i32(E + 1), i32(T, k), i32(R)
    M.mhc_moe_sort(ids, align, *out)
    return out


def random_ids(T, k, E, kind, seed=0):
    g = rng(seed)
    if kind == "one":
        return torch.full((T, k), E - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int32)
    ids = (E * torch.rand(T, k, generator=g) ** 3).int().clamp(max=E - 1)  # skewed, repeats
    return torch.where(torch.rand(T, k, generator=g) < 0.1, -1, ids).int()


@pytest.mark.parametrize("kind", ["skewed", "one", "none"])
@pytest.mark.parametrize("T,k,E,align", [(0, 2, 5, 8), (1, 1, 1, 1), (1, 8, 256, 16), (37, 4, 60, 16),
                                         (511, 2, 7, 1), (1000, 32, 1024, 128), (4097, 8, 61, 64),
                                         (20011, 8, 256, 128), (3, 3, 1000, 65536),
                                         (2000, 32, 1024, 8), (8192, 4, 33, 16), (32769, 1, 2, 4),
                                         (70001, 5, 64, 32)])
def test_sort(M, T, k, E, align, kind):
    ids = random_ids(T, k, E, kind)
    want_rows = M.mhc_moe_rows(T, k, E, align)
    for R in (want_rows, want_rows + 77):
        got = plan(M, ids.cuda(), E, align, R)
        for x, y, n in zip(got, O.sort(ids.numpy(), E, align, R), ("counts", "offsets", "row_of",
                                                                   "slot_of")):
            assert np.array_equal(x.cpu().numpy(), y), n
    assert M.mhc_device_error() == 0


def test_sort_many_slots(M):
    """More slots than one pass of the cluster holds."""
    ids = random_ids(300007, 5, 128, "skewed", 1)
    for x, y in zip(plan(M, ids.cuda(), 128, 128),
                    O.sort(ids.numpy(), 128, 128, M.mhc_moe_rows(300007, 5, 128, 128))):
        assert np.array_equal(x.cpu().numpy(), y)


def test_sort_drops_and_reports_bad_experts(M):
    ids = random_ids(50, 4, 9, "skewed", 2)
    clean = ids.clone()
    for i, bad in enumerate((9, -2, 2 ** 31 - 1, -2 ** 31)):
        ids[i, i], clean[i, i] = bad, -1
    got = plan(M, ids.cuda(), 9, 4)
    assert M.mhc_device_error() == 202 and M.mhc_device_error() == 0
    for x, y in zip(got, plan(M, clean.cuda(), 9, 4)):
        assert torch.equal(x, y)


ROWS = [(1, 1, 1, 1, 8), (1, 8, 256, 8, 7168), (37, 4, 60, 16, 264), (64, 2, 4, 128, 4096),
        (300, 9, 12, 4, 136), (5, 32, 40, 1, 72), (0, 2, 3, 8, 64), (33, 3, 7, 64, 8)]


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("kind", ["skewed", "none"])
@pytest.mark.parametrize("T,k,E,align,C", ROWS)
def test_rows(M, T, k, E, align, C, kind, dt):
    """dispatch and combine, both ways; padding rows hold NaN where they are
    read from and are zeroed where they are written."""
    g = rng(T + C)
    ids = random_ids(T, k, E, kind, C)
    R = M.mhc_moe_rows(T, k, E, align) + 3
    _, _, row_of, slot_of = plan(M, ids.cuda(), E, align, R)
    ro, so = row_of.cpu().numpy(), slot_of.cpu().numpy()
    x = torch.randn(T, C, generator=g).to(dt).cuda()
    xs = torch.full((R, C), 7.0, dtype=dt, device="cuda")
    M.mhc_moe_dispatch_fwd(x, row_of, slot_of, xs)
    if T:
        assert np.array_equal(O.np64(xs), O.dispatch(O.np64(x), so, k))
    else:
        assert torch.all(xs == 0)
    ys = torch.randn(R, C, generator=g).to(dt).cuda()
    ys[slot_of < 0] = float("nan")
    w = torch.rand(T, k, generator=g).cuda()
    df = torch.randn(T, C, generator=g).to(dt).cuda()
    clean = torch.nan_to_num(ys)
    f, dx = (torch.full((T, C), 7.0, dtype=dt, device="cuda") for _ in range(2))
    M.mhc_moe_combine_fwd(ys, w, row_of, f)
    M.mhc_moe_dispatch_bwd(ys, row_of, dx)
    O.check(f, *O.combine(O.np64(clean), O.np64(w), ro), k + 1, "f")
    O.check(dx, *O.combine(O.np64(clean), None, ro), k, "dx")
    dys, dw = torch.full_like(ys, 7), torch.full((T, k), 7.0, device="cuda")
    M.mhc_moe_combine_bwd(df, ys, w, row_of, slot_of, dys, dw)
    if T:
        rys, rdw, rdwm = O.combine_bwd(O.np64(df), O.np64(clean), O.np64(w), ro, so)
        O.check(dys, rys, np.abs(rys), 1, "dys")
        O.check(dw, rdw, rdwm, C, "dw")
    else:
        assert torch.all(dys == 0)
    # weights that are not trained, and no weights
    dys2 = torch.full_like(ys, 7)
    M.mhc_moe_combine_bwd(df, ys, w, row_of, slot_of, dys2, None)
    assert torch.equal(dys2, dys)
    f1, dys1 = torch.empty_like(f), torch.empty_like(ys)
    M.mhc_moe_combine_fwd(ys, None, row_of, f1)
    M.mhc_moe_combine_bwd(df, ys, None, row_of, slot_of, dys1, None)
    M.mhc_moe_dispatch_fwd(df, row_of, slot_of, dys2)
    assert torch.equal(f1, dx) and torch.equal(dys1, dys2)
    assert M.mhc_device_error() == 0


def test_rows_out_of_range_are_left_out_and_reported(M):
    T, k, R, C = 4, 2, 10, 64
    row_of = torch.tensor([[0, 1], [2, 10], [-2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    good = torch.tensor([[0, 1], [2, -1], [-1, 3], [4, 5]], dtype=torch.int32, device="cuda")
    slot_of = torch.tensor([0, 1, 2, 5, 6, 7, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    x, ys = torch.randn(T, C, device="cuda"), torch.randn(R, C, device="cuda")
    w = torch.rand(T, k, device="cuda")

    def calls(plan_rows):
        xs, f, dys, dw = (torch.zeros(s, device="cuda") for s in ((R, C), (T, C), (R, C), (T, k)))
        M.mhc_moe_dispatch_fwd(x, plan_rows, slot_of, xs)
        e = [M.mhc_device_error()]
        M.mhc_moe_combine_fwd(ys, w, plan_rows, f)
        e.append(M.mhc_device_error())
        M.mhc_moe_combine_bwd(x, ys, w, plan_rows, slot_of, dys, dw)
        return [xs, f, dys, dw], e + [M.mhc_device_error()]

    a, ea = calls(row_of)
    b, eb = calls(good)
    assert ea == [203] * 3 and eb == [0] * 3
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_token_does_not_depend_on_the_batch(M):
    T, k, E, C = 700, 4, 16, 520
    g = rng(9)
    ids = random_ids(T, k, E, "skewed", 9).cuda()
    logits = torch.randn(T, 64, generator=g).cuda()
    _, _, row_of, slot_of = plan(M, ids, E, 8)
    ys = torch.randn(slot_of.shape[0], C, generator=g).bfloat16().cuda()
    w, df = torch.rand(T, k, generator=g).cuda(), torch.randn(T, C, generator=g).bfloat16().cuda()
    f, dys, dw = torch.empty_like(df), torch.empty_like(ys), torch.empty_like(w)
    M.mhc_moe_combine_fwd(ys, w, row_of, f)
    M.mhc_moe_combine_bwd(df, ys, w, row_of, slot_of, dys, dw)
    rid, rw = route(M, logits, 8, "softmax", False)
    for t in (0, 333, T - 1):
        s = slice(t, t + 1)
        f1, dw1 = torch.empty_like(df[s]), torch.empty_like(w[s])
        M.mhc_moe_combine_fwd(ys, w[s], row_of[s], f1)
        M.mhc_moe_combine_bwd(df[s].contiguous(), ys, w[s], row_of[s], slot_of, torch.empty_like(ys),
                              dw1)
        i1, w1 = route(M, logits[s], 8, "softmax", False)
        assert torch.equal(f1, f[s]) and torch.equal(dw1, dw[s])
        assert torch.equal(i1, rid[s]) and torch.equal(w1, rw[s])


def test_offsets_past_32_bits(M):
    """Sorted rows of more than 2^31 elements: the last ones are the ones used."""
    T, k, C = 3, 2, 8192
    R = (1 << 31) // C + 64
    row_of = torch.tensor([[R - 1, R - 2], [R - 3, -1], [5, R - 4]], dtype=torch.int32, device="cuda")
    slot_of = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    slot_of[row_of[row_of >= 0].long()] = torch.nonzero(row_of.reshape(-1) >= 0)[:, 0].int()
    x = torch.randn(T, C, generator=rng(1)).bfloat16().cuda()
    xs = torch.full((R, C), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mhc_moe_dispatch_fwd(x, row_of, slot_of, xs)
    used = slot_of >= 0
    assert torch.equal(xs[used], x[(slot_of[used] // k).long()])
    assert torch.count_nonzero(xs[~used][-100:]) == 0 and torch.count_nonzero(xs[:5]) == 0
    f, dw, w = torch.empty_like(x), torch.empty(T, k, device="cuda"), torch.rand(T, k, device="cuda")
    M.mhc_moe_combine_fwd(xs, w, row_of, f)
    ro = row_of.cpu().numpy()
    small = O.dispatch(O.np64(x), np.arange(T * k), k)
    at = np.where(ro >= 0, np.arange(T * k).reshape(T, k), -1)
    O.check(f, *O.combine(small, O.np64(w), at), k + 1, "f")
    dys = torch.full((R, C), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mhc_moe_combine_bwd(x, xs, w, row_of, slot_of, dys, dw)
    _, rdw, rdwm = O.combine_bwd(O.np64(x), small, O.np64(w), at, np.arange(T * k))
    O.check(dw, rdw, rdwm, C, "dw")
    assert torch.count_nonzero(dys[R - 40:R - 5]) == 0 and torch.count_nonzero(dys[R - 1]) > 0


def test_graph_of_the_whole_way(M):
    """Router, sort, dispatch, combine and their gradients captured into one
    graph, replayed on new inputs in the captured tensors; the number of rows
    in use changes between replays."""
    T, k, E, C, align = 190, 4, 24, 136, 16
    g = rng(5)
    R = M.mhc_moe_rows(T, k, E, align)
    bf = torch.bfloat16
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    logits, x = torch.randn(T, E, generator=g).cuda(), torch.randn(T, C, generator=g).to(bf).cuda()
    df = torch.randn(T, C, generator=g).to(bf).cuda()
    o = {"ids": i32(T, k), "w": e(T, k), "counts": i32(E), "offsets": i32(E + 1),
         "row_of": i32(T, k), "slot_of": i32(R), "xs": e(R, C, dt=bf), "f": e(T, C, dt=bf),
         "dys": e(R, C, dt=bf), "dw": e(T, k), "dx": e(T, C, dt=bf), "dl": e(T, E)}

    def step():
        M.mhc_moe_router_fwd(logits, M.SCORE_SOFTMAX, True, 1.0, o["ids"], o["w"])
        M.mhc_moe_sort(o["ids"], align, o["counts"], o["offsets"], o["row_of"], o["slot_of"])
        M.mhc_moe_dispatch_fwd(x, o["row_of"], o["slot_of"], o["xs"])
        M.mhc_moe_combine_fwd(o["xs"], o["w"], o["row_of"], o["f"])
        M.mhc_moe_combine_bwd(df, o["xs"], o["w"], o["row_of"], o["slot_of"], o["dys"], o["dw"])
        M.mhc_moe_dispatch_bwd(o["dys"], o["row_of"], o["dx"])
        M.mhc_moe_router_bwd(o["dw"], logits, o["ids"], M.SCORE_SOFTMAX, True, 1.0, o["dl"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        logits.copy_(torch.randn(T, E, generator=rng(seed)) * seed)
        x.copy_(torch.randn(T, C, generator=rng(seed + 10)))
        for v in o.values():
            v.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in o.items()}
        step()
        for n in o:
            assert torch.equal(got[n], o[n]), n
        # identity experts with weights that sum to 1 give the tokens back
        assert torch.allclose(o["f"].float(), x.float(), atol=0, rtol=2.0 ** -7)
    assert M.mhc_device_error() == 0
