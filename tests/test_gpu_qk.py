"""q/k norm + rotation on the GPU against the plain 64-bit form (tests/_edges.py
says how the tolerances come about)."""
import numpy as np
import pytest
import torch

from tests import _edges as O

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def make(T, Hq, Hk, D, R, dt, seed=0, P=97):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    scale = 0.1 + 3 * torch.rand(T, 1, 1, generator=g)
    d = {"q": (rnd(T, Hq, D) * scale).to(dt), "k": (rnd(T, Hk, D) * scale).to(dt),
         "gq": 1 + 0.2 * rnd(D), "gk": 1 + 0.2 * rnd(D),
         "dq": rnd(T, Hq, D).to(dt), "dk": rnd(T, Hk, D).to(dt),
         "pos": torch.randint(0, P, (T,), generator=g).int()}
    cos, sin = O.rope_table(P, R)
    d["cos"], d["sin"] = torch.from_numpy(cos), torch.from_numpy(sin)
    return {n: v.cuda() for n, v in d.items()}


def table(d):
    at = d["pos"].long().cpu().numpy()
    return O.np64(d["cos"])[at], O.np64(d["sin"])[at]


def run_fwd(M, d, inter, q=None, k=None, qo=None, ko=None):
    q = d["q"] if q is None else q
    k = d["k"] if k is None else k
    qo = torch.full_like(d["q"], 7) if qo is None else qo
    ko = torch.full_like(d["k"], 7) if ko is None else ko
    M.mhc_qk_norm_rope_fwd(q, k, d["gq"], d["gk"], d["cos"], d["sin"], d["pos"], EPS, qo, ko,
                           interleaved=inter)
    return qo, ko


def run_bwd(M, d, inter, dq=None, dk=None, **kw):
    T, Hq, D = d["q"].shape
    Hk = d["k"].shape[1]
    dq = torch.full_like(d["q"], 7) if dq is None else dq
    dk = torch.full_like(d["k"], 7) if dk is None else dk
    dgq, dgk = (torch.full((D,), 7.0, device="cuda") for _ in "qk")
    M.mhc_qk_norm_rope_bwd(kw.get("uq", d["dq"]), kw.get("uk", d["dk"]), kw.get("q", d["q"]),
                           kw.get("k", d["k"]), d["gq"], d["gk"], d["cos"], d["sin"], d["pos"],
                           EPS, dq, dk, dgq, dgk, M.workspace(M.OP_QK_NORM_ROPE_BWD, T, Hq + Hk, D),
                           interleaved=inter)
    return dq, dk, dgq, dgk


# T, Hq, Hk, D, R, interleaved: one token; many heads; every width of vector
# (R of 16: 8; R of 4: 2; else 1); an odd head size; no rotation; no k; the
# largest head; enough work for the walk over tokens
SHAPES = [(1, 32, 8, 128, 128, False), (3, 5, 1, 64, 64, True), (17, 7, 7, 80, 20, False),
          (5, 3, 2, 72, 72, False), (4, 2, 2, 40, 18, False), (6, 3, 1, 33, 10, True),
          (9, 4, 2, 256, 64, True), (2, 1, 1, 512, 512, False), (65, 20, 4, 112, 56, True),
          (3, 2, 1, 8, 0, False), (11, 4, 0, 96, 96, False), (701, 16, 4, 128, 64, False),
          (2051, 4, 1, 72, 16, True), (1, 1, 1, 2, 2, False), (3, 2, 2, 1, 0, False),
          (260, 33, 9, 192, 192, False)]


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", SHAPES)
def test_forward(M, T, Hq, Hk, D, R, inter, dt):
    d = make(T, Hq, Hk, D, R, dt)
    for got, x, g in zip(run_fwd(M, d, inter), ("q", "k"), ("gq", "gk")):
        ref, mag = O.qk_fwd(O.np64(d[x]), O.np64(d[g]), *table(d), R, inter, EPS)
        # rho: the sum of D squares, its root; then gamma and the rotation
        O.check(got, ref, mag, D / 2 + 12, x)
    assert M.mhc_device_error() == 0


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", SHAPES)
def test_backward(M, T, Hq, Hk, D, R, inter, dt):
    d = make(T, Hq, Hk, D, R, dt, seed=1)
    dq, dk, dgq, dgk = run_bwd(M, d, inter)
    for got, gg, x, u, g, H in ((dq, dgq, "q", "dq", "gq", Hq), (dk, dgk, "k", "dk", "gk", Hk)):
        dx, dxm, dg, dgm = O.qk_bwd(O.np64(d[u]), O.np64(d[x]), O.np64(d[g]), *table(d), R, inter,
                                    EPS)
        # rho twice and the sum of D products; dgamma: the sum of T H products of them
        O.check(got, dx, dxm, 2 * D + 20, "d" + x)
        O.check(gg, dg, dgm, T * H + D + 20, "dgamma " + x)
    assert M.mhc_device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,R", [(128, 128), (40, 20)])
def test_layouts_give_the_contiguous_result(M, D, R, dt):
    """Packed qkv views, head-major, broadcast and unaligned inputs and
    outputs, and calls in place."""
    T, Hq, Hk = 37, 6, 2
    d = make(T, Hq, Hk, D, R, dt, seed=2)
    qo, ko = run_fwd(M, d, False)
    dq, dk, dgq, dgk = run_bwd(M, d, False)
    packed = torch.full((T, Hq + 2 * Hk, D), 9.0, dtype=dt, device="cuda")
    packed[:, :Hq], packed[:, Hq:Hq + Hk] = d["q"], d["k"]
    pq, pk = packed[:, :Hq], packed[:, Hq:Hq + Hk]
    hq = torch.empty(Hq, T, D, dtype=dt, device="cuda")
    hk = torch.empty(Hk, T, D, dtype=dt, device="cuda")
    a, b = run_fwd(M, d, False, pq, pk, hq.transpose(0, 1), hk.transpose(0, 1))
    assert torch.equal(a, qo) and torch.equal(b, ko)
    got = run_bwd(M, d, False, hq.transpose(0, 1), hk.transpose(0, 1), q=pq, k=pk)
    for x, y in zip(got, (dq, dk, dgq, dgk)):
        assert torch.equal(x, y)
    # in place: the packed product itself, then the gradients over the upstream ones
    run_fwd(M, d, False, pq, pk, pq, pk)
    assert torch.equal(pq, qo) and torch.equal(pk, ko)
    assert torch.all(packed[:, Hq + Hk:] == 9)
    uq, uk = d["dq"].clone(), d["dk"].clone()
    run_bwd(M, d, False, uq, uk, uq=uq, uk=uk)
    assert torch.equal(uq, dq) and torch.equal(uk, dk)
    # one element off: another vector width, so the sums' order may differ
    off = torch.empty(T * Hq * D + 1, dtype=dt, device="cuda")[1:].view(T, Hq, D)
    off.copy_(d["q"])
    a, _ = run_fwd(M, d, False, off, None, torch.empty_like(off), None)
    ref, mag = O.qk_fwd(O.np64(d["q"]), O.np64(d["gq"]), *table(d), R, False, EPS)
    O.check(a, ref, mag, D / 2 + 12, "unaligned")
    # one row for all tokens and heads
    row = d["q"][:1, :1].expand(T, Hq, D)
    a, _ = run_fwd(M, d, False, row)
    ref, mag = O.qk_fwd(O.np64(row), O.np64(d["gq"]), *table(d), R, False, EPS)
    O.check(a, ref, mag, D / 2 + 12, "broadcast")


# long inputs (the walk over tokens): the largest head, heads that fill their
# lanes and heads that do not, more heads than lanes, both pairings
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", [
    (2500, 3, 1, 512, 512, False), (2450, 4, 0, 64, 64, True), (203, 70, 5, 16, 16, False),
    (611, 14, 2, 96, 96, True), (305, 33, 0, 256, 256, False), (1300, 7, 1, 128, 48, False),
    (401, 24, 3, 80, 20, False)])
def test_long_inputs_in_any_layout(M, T, Hq, Hk, D, R, inter, dt):
    d = make(T, Hq, Hk, D, R, dt, seed=8)
    d["pos"][T // 2] = 97  # one token without a place in the table
    qo, ko = run_fwd(M, d, inter)
    dq, dk, dgq, dgk = run_bwd(M, d, inter)
    assert M.mhc_device_error() == 201
    at = d["pos"].long().cpu().numpy()
    cos, sin = (O.np64(d[n])[np.minimum(at, 96)] for n in ("cos", "sin"))
    keep = np.arange(T) != T // 2
    for y, gy, gg, x, u, g, H in ((qo, dq, dgq, "q", "dq", "gq", Hq), (ko, dk, dgk, "k", "dk", "gk", Hk)):
        args = O.np64(d[x])[keep], O.np64(d[g]), cos[keep], sin[keep], R, inter, EPS
        assert torch.all(y[T // 2] == 0) and torch.all(gy[T // 2] == 0)
        k = torch.from_numpy(keep).cuda()
        O.check(y[k], *O.qk_fwd(*args), D / 2 + 12, x)
        dx, dxm, dg, dgm = O.qk_bwd(O.np64(d[u])[keep], *args)
        O.check(gy[k], dx, dxm, 2 * D + 20, "d" + x)
        O.check(gg, dg, dgm, T * H + D + 20, "dgamma " + x)
    # head-major inputs and outputs
    major = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    e = dict(d, **{n: major(d[n]) for n in ("q", "k", "dq", "dk")})
    a, b = run_fwd(M, e, inter, qo=major(qo), ko=major(ko))
    assert torch.equal(a, qo) and torch.equal(b, ko)
    for x, y in zip(run_bwd(M, e, inter, major(dq), major(dk)), (dq, dk, dgq, dgk)):
        assert torch.equal(x, y)
    M.mhc_device_error()


def test_no_gamma_no_positions_no_rotation_no_k(M):
    d = make(5, 3, 2, 64, 64, torch.bfloat16, seed=3)
    plain = dict(d, gq=None, gk=None, pos=None)
    ones = dict(d, gq=torch.ones(64, device="cuda"), gk=torch.ones(64, device="cuda"),
                pos=torch.arange(5, dtype=torch.int32, device="cuda"))
    for x, y in zip(run_fwd(M, plain, False), run_fwd(M, ones, False)):
        assert torch.equal(x, y)
    for x, y in zip(run_bwd(M, plain, False), run_bwd(M, ones, False)):
        assert torch.equal(x, y)
    # cos and sin None: the norm alone, the rotation by angle 0
    still = dict(d, cos=torch.ones_like(d["cos"]), sin=torch.zeros_like(d["sin"]))
    for x, y in zip(run_fwd(M, dict(d, cos=None, sin=None), False), run_fwd(M, still, False)):
        assert torch.equal(x, y)
    qo = torch.empty_like(d["q"])
    M.mhc_qk_norm_rope_fwd(d["q"], None, d["gq"], None, d["cos"], d["sin"], d["pos"], EPS, qo, None)
    assert torch.equal(qo, run_fwd(M, d, False)[0])
    # gammas that are not trained need no workspace
    dq, dk = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    M.mhc_qk_norm_rope_bwd(d["dq"], d["dk"], d["q"], d["k"], d["gq"], d["gk"], d["cos"], d["sin"],
                           d["pos"], EPS, dq, dk)
    assert torch.equal(dq, run_bwd(M, d, False)[0]) and torch.equal(dk, run_bwd(M, d, False)[1])


@pytest.mark.parametrize("D,R", [(128, 128), (80, 20), (33, 2)])
def test_zero_rows_bad_positions_and_empty(M, D, R):
    d = make(6, 2, 1, D, R, torch.bfloat16, seed=4)
    d["q"][2] = 0
    out = torch.empty_like(d["q"])
    M.mhc_qk_norm_rope_fwd(d["q"], None, d["gq"], None, d["cos"], d["sin"], d["pos"], 0.0, out,
                           None)
    assert torch.all(out[2] == 0) and torch.all(torch.isfinite(out))
    good, goodb = run_fwd(M, d, False), run_bwd(M, d, False)
    assert M.mhc_device_error() == 0
    for bad in (-1, 97):
        e = dict(d, pos=d["pos"].clone())
        e["pos"][3] = bad
        got, gotb = run_fwd(M, e, False), run_bwd(M, e, False)
        assert M.mhc_device_error() == 201 and M.mhc_device_error() == 0
        keep = [0, 1, 2, 4, 5]
        for x, y in zip(got + gotb[:2], good + goodb[:2]):
            assert torch.equal(x[keep], y[keep]) and torch.all(x[3] == 0)
    # no tokens: the sums over them are zero
    none = {n: (v[:0] if n in ("q", "k", "dq", "dk", "pos") else v) for n, v in d.items()}
    _, _, dgq, dgk = run_bwd(M, none, False)
    assert torch.all(dgq == 0) and torch.all(dgk == 0)
    run_fwd(M, none, False)


def test_a_token_does_not_depend_on_the_batch(M):
    """A long batch (several heads to a warp, a walk over tokens), a short one
    and a single token give the same bits; so does a second run."""
    T = 900
    d = make(T, 16, 4, 128, 128, torch.bfloat16, seed=5)
    qo, ko = run_fwd(M, d, False)
    dq, dk, dgq, dgk = run_bwd(M, d, False)
    for t in (0, 413, T - 1):
        one = {n: (v[t:t + 1] if n in ("q", "k", "dq", "dk", "pos") else v) for n, v in d.items()}
        a, b = run_fwd(M, one, False)
        x, y, _, _ = run_bwd(M, one, False)
        assert torch.equal(a, qo[t:t + 1]) and torch.equal(b, ko[t:t + 1])
        assert torch.equal(x, dq[t:t + 1]) and torch.equal(y, dk[t:t + 1])
    for x, y in zip(run_bwd(M, d, False), (dq, dk, dgq, dgk)):
        assert torch.equal(x, y)


def test_long_backward_repeats_bit_for_bit(M):
    """The rings' slots are refilled while others are read."""
    d = make(4096, 32, 8, 128, 128, torch.bfloat16, seed=9, P=4096)
    first = run_bwd(M, d, False)
    for _ in range(100):
        assert all(torch.equal(x, y) for x, y in zip(run_bwd(M, d, False), first))


def test_offsets_past_32_bits(M):
    """Token strides that put the last token more than 2^32 bytes away."""
    step, T, H, D = (1 << 30) + 64, 3, 2, 64
    big = torch.empty((T - 1) * step + H * D, dtype=torch.bfloat16, device="cuda")
    view = big.as_strided((T, H, D), (step, D, 1))
    d = make(T, H, H, D, D, torch.bfloat16, seed=6)
    qo, _ = run_fwd(M, d, False)
    view.copy_(d["q"])
    a, _ = run_fwd(M, d, False, view, None, view, None)
    assert torch.equal(a, qo)


def test_graph_and_side_stream(M):
    d = make(33, 8, 2, 128, 128, torch.bfloat16, seed=7)
    want = run_bwd(M, d, False)
    got = [torch.zeros_like(x) for x in want]
    ws = M.workspace(M.OP_QK_NORM_ROPE_BWD, 33, 10, 128)
    call = lambda s=None: M.mhc_qk_norm_rope_bwd(  # noqa: E731
        d["dq"], d["dk"], d["q"], d["k"], d["gq"], d["gk"], d["cos"], d["sin"], d["pos"], EPS,
        *got, ws, stream=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in got:
        x.zero_()
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    d["dq"].neg_()
    g.replay()
    assert torch.equal(got[0], -want[0]) and torch.equal(got[2], -want[2])
