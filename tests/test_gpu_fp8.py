"""The 8-bit floating-point operators against plain forms: quantisation to the
bit, the rest against 64 bits (tests/_fp8.py says how the tolerances come about)."""
import math

import numpy as np
import pytest
import torch

from tests import _fp8 as F8
from tests._edges import DTYPES, U, check, np64
from tests._fp8 import E4M3, E5M2, blocks

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    yield m
    assert m.mhc_device_error() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(R, C, seed, dtype=torch.float32):
    g = gen(seed)
    x = torch.randn(R, C, generator=g) * (0.1 + 3 * torch.rand(R, 1, generator=g))
    return x.to(dtype)


def full(*shape, dtype=torch.float32):
    """An output full of what a result must not be."""
    return torch.full(shape, math.nan, device="cuda").to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int32).cpu()


def outputs(G, R, C, fmt, tiles, which):
    lead = (G,) if G else ()
    q = s = qt = st = None
    if "q" in which:
        q, s = full(*lead, R, C, dtype=fmt), full(*lead, blocks(C), blocks(R) if tiles else R)
    if "t" in which:
        qt, st = full(*lead, C, R, dtype=fmt), full(*lead, blocks(R), blocks(C) if tiles else C)
    return q, s, qt, st


@pytest.mark.parametrize("R,C,which", [(1, 16, "q"), (37, 7168, "q"), (130, 144, "q"), (16, 16, "qt"),
                                       (144, 400, "qt"), (256, 256, "qt"), (272, 1328, "t")])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quant_to_the_bit(M, R, C, which, fmt, dtype):
    x = rows(R, C, R + C, dtype)
    q, s, qt, st = outputs(0, R, C, fmt, False, which)
    M.mhc_fp8_quant(x.cuda(), q, s, qt, st)
    for got, ref in ((q, s), F8.quant_rows(x.float(), fmt)), ((qt, st), F8.quant_rows(x.float().t(), fmt)):
        if got[0] is not None:
            assert torch.equal(bits(got[0]), bits(ref[0])) and torch.equal(bits(got[1]), bits(ref[1]))


@pytest.mark.parametrize("G,R,C", [(0, 16, 16), (0, 272, 144), (3, 144, 400), (2, 128, 256)])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_quant_tiles_to_the_bit(M, G, R, C, fmt):
    x = rows(max(G, 1) * R, C, R + C, torch.bfloat16)
    x = x.reshape(G, R, C) if G else x
    q, s, qt, st = outputs(G, R, C, fmt, True, "qt")
    M.mhc_fp8_quant(x.cuda(), q, s, qt, st, tiles=True)
    rq, rs = F8.quant_tiles(x.float(), fmt)
    assert torch.equal(bits(q), bits(rq)) and torch.equal(bits(s), bits(rs))
    assert torch.equal(bits(qt), bits(rq.transpose(-1, -2))) and torch.equal(bits(st), bits(rs.transpose(-1, -2)))


def test_quant_small_large_and_not_numbers(M):
    """Blocks of zeros, of subnormals, of the largest numbers; an infinity or a NaN is its
    block's alone."""
    x = rows(32, 640, 5)
    x[3, :128] = 0
    x[4, 128:256] = 1e-42
    x[5, :128] *= 1e37
    x[6, 256:384] = 2.0 ** -101
    x[7, 130], x[8, 400], x[9, 639] = math.inf, math.nan, -math.inf
    q, s, qt, st = outputs(0, 32, 640, E4M3, False, "qt")
    M.mhc_fp8_quant(x.cuda(), q, s, qt, st)
    rq, rs = F8.quant_rows(x, E4M3)
    bad = torch.zeros(5, 32, dtype=torch.bool)
    bad[1, 7] = bad[3, 8] = bad[4, 9] = True
    assert torch.equal(s.cpu().isnan(), bad)
    assert torch.equal(s.cpu()[~bad], rs[~bad])
    keep = (~bad).t().repeat_interleave(128, 1)
    assert torch.equal(bits(q)[keep], bits(rq)[keep])
    cols = torch.zeros(640, dtype=torch.bool)
    cols[[130, 400, 639]] = True
    assert torch.equal(st.cpu()[0].isnan(), cols)
    assert F8.values(q, s)[3, :128].tolist() == [0.0] * 128


def test_quant_ties(M):
    """Values halfway between two of the format go to the even one; a block's largest is exact."""
    v = torch.tensor([448.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 416.0 + 16, -1.0625, 0.0])
    x = v.repeat(16)[None].repeat(16, 1)
    q, s, _, _ = outputs(0, 16, 128, E4M3, False, "q")
    M.mhc_fp8_quant(x.cuda(), q, s)
    assert np64(s)[0].tolist() == [1.0] * 16
    assert q.cpu().float()[0, :8].tolist() == [448.0, 1.0, 1.25, 0.0, 2.0 ** -8, 448.0, -1.0, 0.0]


@pytest.mark.parametrize("R,F", [(16, 16), (144, 208), (272, 128), (130, 400)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_swiglu(M, R, F, dtype, fmt):
    h, da = rows(R, 2 * F, R, dtype), rows(R, F, R + 1, dtype)
    h[0, :F] = torch.linspace(-60, 60, F).to(dtype)
    both = "qt" if R % 16 == 0 else "q"
    for way in ("fwd", "bwd"):
        C = F if way == "fwd" else 2 * F
        y = full(R, C, dtype=dtype)
        q, s, qt, st = outputs(0, R, C, fmt, False, both)
        if way == "fwd":
            M.mhc_fp8_swiglu_fwd(h.cuda(), y, q, s, qt, st)
            ref, err = F8.swiglu(np64(h))
        else:
            M.mhc_fp8_swiglu_bwd(da.cuda(), h.cuda(), y, q, s, qt, st)
            ref, err = F8.swiglu_grad(np64(da), np64(h))
        check(y, ref, err / U, 1.0, way)
        F8.check_quantised(q, s, ref, err, way + " rows")
        if qt is not None:
            F8.check_quantised(qt, st, ref.T.copy(), err.T.copy(), way + " columns")
        only = full(R, C, dtype=dtype)  # the values alone
        if way == "fwd":
            M.mhc_fp8_swiglu_fwd(h.cuda(), only)
        else:
            M.mhc_fp8_swiglu_bwd(da.cuda(), h.cuda(), only)
        assert torch.equal(only, y)


@pytest.mark.parametrize("F", [1024, 1040])
@pytest.mark.parametrize("which", ["q", "t", "qt"])
def test_of_more_tiles_than_run_at_a_time(M, F, which):
    """A block goes through several tiles, the gate's and up's of them in pairs or one by one."""
    R = 5008
    h, da = rows(R, 2 * F, F, torch.bfloat16), rows(R, F, F + 1, torch.bfloat16)
    q, s, qt, st = outputs(0, R, 2 * F, E4M3, False, which)
    M.mhc_fp8_quant(h.cuda(), q, s, qt, st)
    for got, ref in ((q, s), F8.quant_rows(h.float(), E4M3)), ((qt, st), F8.quant_rows(h.float().t(), E4M3)):
        if got[0] is not None:
            assert torch.equal(bits(got[0]), bits(ref[0])) and torch.equal(bits(got[1]), bits(ref[1]))
    for way, ref, err in ("fwd", *F8.swiglu(np64(h))), ("bwd", *F8.swiglu_grad(np64(da), np64(h))):
        C = ref.shape[1]
        for y in (None, full(R, C, dtype=torch.bfloat16)):
            q, s, qt, st = outputs(0, R, C, E4M3, False, which)
            if way == "fwd":
                M.mhc_fp8_swiglu_fwd(h.cuda(), y, q, s, qt, st)
            else:
                M.mhc_fp8_swiglu_bwd(da.cuda(), h.cuda(), y, q, s, qt, st)
            if y is not None:
                check(y, ref, err / U, 1.0, way)
            if q is not None:
                F8.check_quantised(q, s, ref, err, way + " rows")
            if qt is not None:
                F8.check_quantised(qt, st, ref.T.copy(), err.T.copy(), way + " columns")


def test_swiglu_gradient_against_differences(M):
    R, F, d = 16, 32, 2.0 ** -7
    h, da = rows(R, 2 * F, 1), rows(R, F, 2)
    dh = full(R, 2 * F)
    M.mhc_fp8_swiglu_bwd(da.cuda(), h.cuda(), dh)
    h64, da64 = np64(h), np64(da)
    err = F8.swiglu_grad(da64, h64)[1]
    for c in range(2 * F):
        step = np.zeros(2 * F)
        step[c] = d
        diff = ((F8.swiglu(h64 + step)[0] - F8.swiglu(h64 - step)[0]) * da64).sum(1) / (2 * d)
        # a central difference is off by d^2 / 6 of a third derivative, here below |da up|
        tol = d * d / 6 * np.abs(da64 * h64[:, F:]).max(1) + err[:, c] + 2.0 ** -24 * np.abs(diff)
        assert np.all(np.abs(np64(dh)[:, c] - diff) <= tol + 1e-9)


def test_swiglu_infinite_gate(M):
    """A gate of -inf gives 0 and a gradient of 0, as the limits are."""
    h = torch.zeros(16, 32)
    h[:, :16], h[:, 16:] = -math.inf, 3.0
    a, dh = full(16, 16), full(16, 32)
    M.mhc_fp8_swiglu_fwd(h.cuda(), a)
    M.mhc_fp8_swiglu_bwd(torch.ones(16, 16).cuda(), h.cuda(), dh)
    assert not a.any() and not dh.any()


# ---- products ---------------------------------------------------------------

def gemm_case(counts, align, N, K, fa, fb, seed, extra=0, garbage=True):
    G = len(counts)
    off = F8.segments(counts, align)
    R = int(off[-1]) + extra
    a, sa = F8.quant_rows(rows(max(R, 1), K, seed)[:R], fa)
    b, sb = F8.quant_tiles(rows(G * N, K, seed + 1).reshape(G, N, K) * K ** -0.5, fb)
    if garbage:  # rows of no segment
        sa[:, int(off[-1]):] = math.nan
    return a, sa, b, sb, off, R


def gemm_ref(a, sa, b, sb, off):
    av, bv, o = F8.values(a, torch.nan_to_num(sa)), F8.values(b, sb), off.tolist()
    ref, mag = np.zeros((a.shape[0], b.shape[1])), np.zeros((a.shape[0], b.shape[1]))
    for e, (lo, hi) in enumerate(zip(o, o[1:])):
        ref[lo:hi] = av[lo:hi] @ bv[e].T
        mag[lo:hi] = np.abs(av[lo:hi]) @ np.abs(bv[e]).T
    return ref, mag


@pytest.mark.parametrize("counts,align,N,K,extra", [
    ([1], 1, 8, 16, 0),                          # the smallest
    ([1], 1, 264, 144, 3),
    ([5, 0, 130, 1], 1, 400, 272, 7),            # segments off every tile, one empty
    ([0, 0, 0], 1, 136, 128, 40),                # nothing at all
    ([129, 64, 300], 16, 1328, 1040, 0),
    ([128, 256], 128, 256, 512, 256),
    ([3000], 8, 520, 384, 0),                    # more row tiles than a group of them
    ([1] * 40, 8, 128, 256, 5),
])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)])
def test_gemm(M, counts, align, N, K, extra, fa, fb):
    a, sa, b, sb, off, R = gemm_case(counts, align, N, K, fa, fb, N + K, extra)
    ref, mag = gemm_ref(a, sa, b, sb, off)
    for dtype in DTYPES:
        out = full(R, N, dtype=dtype)
        M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), out)
        check(out, ref, mag, F8.product_ops(K), str(dtype))


@pytest.mark.parametrize("counts,align,N,K,extra", [
    ([1500, 0, 900, 131], 1, 2824, 272, 5),      # enough tiles for the wider form, odd ends
    ([100] * 24, 8, 1536, 144, 0),               # below 160 rows a segment, whole tiles
    ([5000], 16, 2056, 128, 100),                # one block; more row tiles than two groups
])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3)])
def test_gemm_of_many_tiles(M, counts, align, N, K, extra, fa, fb):
    """And some of the rows in a small call of their own have the bits that they have here."""
    a, sa, b, sb, off, R = gemm_case(counts, align, N, K, fa, fb, N + K, extra)
    ref, mag = gemm_ref(a, sa, b, sb, off)
    dev = [t.cuda() for t in (a, sa, b, sb, off)]
    for dtype in DTYPES:
        out = full(R, N, dtype=dtype)
        M.mhc_fp8_gemm(*dev, out)
        check(out, ref, mag, F8.product_ops(K), str(dtype))
    hi = int(off[-1])
    lo = hi - 90
    few = full(90, N)
    own = dev[1][:, lo:hi].clone(memory_format=torch.contiguous_format)
    M.mhc_fp8_gemm(dev[0][lo:hi], own, dev[2][-1:], dev[3][-1:].clone(), None, few)
    assert torch.equal(few, out[lo:hi])


def test_gemm_many_experts(M):
    """As many as are allowed, most of them without a row."""
    counts = [3 if e % 7 == 0 else 0 for e in range(1024)]
    a, sa, b, sb, off, R = gemm_case(counts, 1, 16, 32, E4M3, E4M3, 1)
    out = full(R, 16)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), out)
    check(out, *gemm_ref(a, sa, b, sb, off), F8.product_ops(32))


def test_gemm_plain_is_one_segment(M):
    a, sa, b, sb, off, R = gemm_case([300], 1, 264, 400, E4M3, E4M3, 9)
    one, other = full(R, 264), full(R, 264)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), None, one)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), other)
    assert torch.equal(one, other)
    check(one, *gemm_ref(a, sa, b, sb, off), F8.product_ops(400))


def test_gemm_rows_do_not_depend_on_the_others(M):
    """A row has the same bits alone and among others, and a NaN stays in its row."""
    a, sa, b, sb, off, R = gemm_case([200, 77], 1, 264, 640, E4M3, E4M3, 4)
    out = full(R, 264)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), out)
    one = full(1, 264)
    M.mhc_fp8_gemm(a[205:206].cuda(), sa[:, 205:206].contiguous().cuda(), b[1:].cuda(), sb[1:].cuda(),
                   None, one)
    assert torch.equal(one[0], out[205])
    sa[2, 100] = math.nan
    again = full(R, 264)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), off.cuda(), again)
    assert again[100].isnan().all()
    assert torch.equal(torch.cat((again[:100], again[101:])), torch.cat((out[:100], out[101:])))


def wgrad_case(counts, M_, N, fa, fb, seed, extra=0):
    off = F8.segments(counts, 128)
    R = int(off[-1]) + extra
    x, y = torch.zeros(R, M_), torch.zeros(R, N)
    for lo, n in zip(off.tolist(), counts):
        x[lo:lo + n], y[lo:lo + n] = rows(n, M_, seed + lo), rows(n, N, seed + lo + 1)
    at, sat = F8.quant_rows(x.t().contiguous(), fa)
    bt, sbt = F8.quant_rows(y.t().contiguous(), fb)
    sat[int(off[-1]) // 128:] = math.nan
    return at, sat, bt, sbt, off


def wgrad_ref(at, sat, bt, sbt, off):
    a, b, o = F8.values(at, torch.nan_to_num(sat)), F8.values(bt, sbt), off.tolist()
    segs = [slice(lo, hi) for lo, hi in zip(o, o[1:])]
    return (np.stack([a[:, s] @ b[:, s].T for s in segs]),
            np.stack([np.abs(a[:, s]) @ np.abs(b[:, s]).T for s in segs]))


@pytest.mark.parametrize("counts,M_,N,extra", [
    ([1], 1, 8, 0), ([0, 5, 0], 130, 264, 128), ([128, 700], 256, 256, 0), ([300], 1000, 400, 0),
    ([1, 0, 2, 129, 40], 72, 1328, 0)])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3)])
def test_wgrad(M, counts, M_, N, extra, fa, fb):
    case = wgrad_case(counts, M_, N, fa, fb, M_, extra)
    ref, mag = wgrad_ref(*case)
    for dtype in DTYPES:
        out = full(len(counts), M_, N, dtype=dtype)
        M.mhc_fp8_wgrad(*(t.cuda() for t in case), out)
        check(out, ref, mag, F8.product_ops(max(counts) + 1), str(dtype))


@pytest.mark.parametrize("counts,M_,N,extra", [
    ([130, 0, 300, 1], 1000, 2824, 128), ([40] * 30, 136, 1536, 0)])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3)])
def test_wgrad_of_many_tiles(M, counts, M_, N, extra, fa, fb):
    case = wgrad_case(counts, M_, N, fa, fb, M_, extra)
    ref, mag = wgrad_ref(*case)
    for dtype in DTYPES:
        out = full(len(counts), M_, N, dtype=dtype)
        M.mhc_fp8_wgrad(*(t.cuda() for t in case), out)
        check(out, ref, mag, F8.product_ops(max(counts) + 1), str(dtype))


def test_wgrad_ragged_last_block_and_plain(M):
    """One segment of rows that are no whole blocks: 128 + 48."""
    x, y = rows(176, 24, 1), rows(176, 40, 2)
    at, sat = F8.quant_rows(x.t().contiguous(), E4M3)
    bt, sbt = F8.quant_rows(y.t().contiguous(), E4M3)
    off = torch.tensor([0, 176], dtype=I32)
    ref, mag = wgrad_ref(at, sat, bt, sbt, off)
    for o in (None, off.cuda()):
        out = full(1, 24, 40)
        M.mhc_fp8_wgrad(at.cuda(), sat.cuda(), bt.cuda(), sbt.cuda(), o, out)
        check(out, ref, mag, F8.product_ops(176))


def test_wgrad_of_no_rows_is_zero(M):
    out = full(2, 16, 24)
    e = torch.empty(16, 0, dtype=E4M3, device="cuda")
    M.mhc_fp8_wgrad(e, torch.empty(0, 16, device="cuda"), torch.empty(24, 0, dtype=E4M3, device="cuda"),
                    torch.empty(0, 24, device="cuda"), torch.zeros(3, dtype=I32, device="cuda"), out)
    assert not out.any()


def test_bad_offsets_are_moved_and_reported(M):
    a, sa, b, sb, _, R = gemm_case([100, 60, 40], 1, 64, 128, E4M3, E4M3, 3)
    for bad, as_if in (([0, 100, 90, 200], [0, 100, 100, 200]), ([-5, 100, 160, 999], [0, 100, 160, 200]),
                       ([10, 100, 160, 190], None)):
        out = full(R, 64)
        M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), torch.tensor(bad, dtype=I32).cuda(), out)
        assert M.mhc_device_error() == (205 if as_if else 0)
        check(out, *gemm_ref(a, sa, b, sb, torch.tensor(as_if or bad)), F8.product_ops(128))
    case = wgrad_case([128, 200], 40, 64, E4M3, E4M3, 1)
    out = full(2, 40, 64)
    off = torch.tensor([0, 130, 384], dtype=I32)
    M.mhc_fp8_wgrad(*(t.cuda() for t in case[:4]), off.cuda(), out)
    assert M.mhc_device_error() == 206
    check(out, *wgrad_ref(*case[:4], torch.tensor([0, 128, 384])), F8.product_ops(256))


# ---- the whole layer for a few tokens ----------------------------------------

def few_case(T, C, F, E, k, dtype, eight, seed, drop=0.1):
    g = gen(seed)
    x = rows(T, C, seed, dtype)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(I32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    w = torch.rand(T, k, generator=g) + 0.05
    w1 = rows(E * 2 * F, C, seed + 1).reshape(E, 2 * F, C) * C ** -0.5
    w2 = rows(E * C, F, seed + 2).reshape(E, C, F) * F ** -0.5
    if eight:
        return x, ids, w, *F8.quant_tiles(w1, E4M3), *F8.quant_tiles(w2, E4M3)
    return x, ids, w, w1.to(dtype), None, w2.to(dtype), None


def few_run(M, case, ws=None):
    x, ids, w, w1, s1, w2, s2 = (None if t is None else t.cuda() for t in case)
    T, C = x.shape
    f = full(T, C, dtype=x.dtype)
    if ws is None:
        ws = M.workspace(M.OP_MOE_FEW_FWD, T, ids.shape[1], C + w2.shape[2])
        ws.fill_(255)  # NaN, and counts that are far off
    M.mhc_moe_few_fwd(x, ids, w, w1, w2, f, ws, s1, s2)
    return f


def few_ref(case):
    x, ids, w, w1, s1, w2, s2 = case
    if s1 is None:
        return F8.few(np64(x), ids.numpy(), np64(w), np64(w1), np64(w2), False)
    xq = F8.values(*F8.quant_rows(x.float(), E4M3))
    return F8.few(xq, ids.numpy(), np64(w), F8.values(w1, s1), F8.values(w2, s2), True)


@pytest.mark.parametrize("T,C,F,E,k", [
    (1, 16, 16, 1, 1), (1, 256, 128, 8, 8), (3, 144, 80, 5, 2), (8, 400, 272, 16, 4), (9, 1040, 144, 4, 2),
    (17, 272, 400, 6, 3), (64, 128, 48, 2, 2), (128, 80, 64, 3, 1), (40, 48, 1040, 32, 8)])
@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("eight", [False, True])
def test_few(M, T, C, F, E, k, dtype, eight):
    case = few_case(T, C, F, E, k, dtype, eight, T + C + F)
    F8.check_few(few_run(M, case), *few_ref(case))


@pytest.mark.parametrize("T,E,k", [(128, 1024, 32), (128, 1023, 32), (128, 4, 4), (5, 1024, 1), (1, 33, 32)])
@pytest.mark.parametrize("eight", [False, True])
def test_few_most_slots_and_experts(M, T, E, k, eight):
    case = few_case(T, 32, 16, E, k, torch.bfloat16, eight, T + E)
    F8.check_few(few_run(M, case), *few_ref(case))


@pytest.mark.parametrize("eight", [False, True])
def test_few_drops_twins_and_strangers(M, eight):
    """No slot at all, an expert named twice by a token, ids outside."""
    x, ids, w, w1, s1, w2, s2 = few_case(12, 160, 96, 4, 3, torch.bfloat16, eight, 3)
    none = torch.full_like(ids, -1)
    assert not few_run(M, (x, none, w, w1, s1, w2, s2)).any()
    twins = torch.zeros_like(ids)  # 36 slots of one expert
    twins[::2, 1] = 2
    case = (x, twins, w, w1, s1, w2, s2)
    F8.check_few(few_run(M, case), *few_ref(case))
    strange = twins.clone()
    strange[3, 0], strange[5, 2] = 4, -7
    out = few_run(M, (x, strange, w, w1, s1, w2, s2))
    assert M.mhc_device_error() == 202
    strange[3, 0] = strange[5, 2] = -1
    assert torch.equal(out, few_run(M, (x, strange, w, w1, s1, w2, s2)))


@pytest.mark.parametrize("eight", [False, True])
def test_few_tokens_do_not_depend_on_the_others(M, eight):
    """The same bits run to run, and (a NaN in one token aside) for the other tokens."""
    x, ids, w, w1, s1, w2, s2 = few_case(24, 400, 144, 6, 2, torch.bfloat16, eight, 8, 0.0)
    out = few_run(M, (x, ids, w, w1, s1, w2, s2))
    for _ in range(5):
        assert torch.equal(out, few_run(M, (x, ids, w, w1, s1, w2, s2)))
    x[7, 3] = math.nan
    again = few_run(M, (x, ids, w, w1, s1, w2, s2))
    assert again[7].isnan().all()
    keep = torch.arange(24) != 7
    assert torch.equal(again[keep.cuda()], out[keep.cuda()])


def test_few_fp16_activation_past_the_type(M):
    """An activation above fp16's largest value is kept (two terms cannot: it is infinite) without
    turning into a NaN by itself."""
    x = torch.ones(1, 16, dtype=torch.float16)
    w1 = torch.full((1, 32, 16), 20.0, dtype=torch.float16)  # gate = up = 320, h = 102400
    w2 = torch.full((1, 16, 16), 1.0, dtype=torch.float16)
    f = few_run(M, (x, torch.zeros(1, 1, dtype=I32), torch.ones(1, 1), w1, None, w2, None))
    assert torch.isinf(f).all()


# ---- together, streams, graphs ----------------------------------------------

def test_few_is_the_sorted_chain(M):
    """Router's choice -> sort -> dispatch -> quantise -> product -> activation -> product ->
    combine against the one call, 8-bit weights, fp32 between the steps."""
    T, C, F, E, k = 48, 400, 272, 8, 3
    x, _, _, w1, s1, w2, s2 = few_case(T, C, F, E, k, torch.bfloat16, True, 21)
    logits = torch.randn(T, E, generator=gen(2)).cuda()
    ids, w = torch.empty(T, k, dtype=I32, device="cuda"), full(T, k)
    M.mhc_moe_router_fwd(logits, M.SCORE_SOFTMAX, True, 1.0, ids, w)
    R = M.mhc_moe_rows(T, k, E, 16)
    cnt, off = torch.empty(E, dtype=I32, device="cuda"), torch.empty(E + 1, dtype=I32, device="cuda")
    row, slot = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(R, dtype=I32, device="cuda")
    M.mhc_moe_sort(ids, 16, cnt, off, row, slot)
    xs = full(R, C, dtype=torch.bfloat16)
    M.mhc_moe_dispatch_fwd(x.cuda(), row, slot, xs)
    q, s = full(R, C, dtype=E4M3), full(blocks(C), R)
    M.mhc_fp8_quant(xs, q, s)
    h = full(R, 2 * F)
    M.mhc_fp8_gemm(q, s, w1.cuda(), s1.cuda(), off, h)
    aq, as_ = full(R, F, dtype=E4M3), full(blocks(F), R)
    M.mhc_fp8_swiglu_fwd(h, None, aq, as_)
    y = full(R, C)
    M.mhc_fp8_gemm(aq, as_, w2.cuda(), s2.cuda(), off, y)
    f = full(T, C)
    M.mhc_moe_combine_fwd(y, w, row, f)
    case = (x, ids.cpu(), w.cpu(), w1, s1, w2, s2)
    ref, err = few_ref(case)
    F8.check_few(f.bfloat16(), ref, err + 2.0 ** -9 * 2.0 ** -15 * np.abs(ref))
    F8.check_few(few_run(M, case), ref, err)


def moe_step(M, p, stream=None):
    """Forward and backward of the experts on sorted rows; p: tensors of one step, outputs among
    them."""
    kw = {"stream": stream}
    M.mhc_fp8_quant(p["xs"], p["xq"], p["xqs"], p["xt"], p["xts"], **kw)
    M.mhc_fp8_gemm(p["xq"], p["xqs"], p["w1"], p["s1"], p["off"], p["h"], **kw)
    M.mhc_fp8_swiglu_fwd(p["h"], None, p["aq"], p["aqs"], p["at"], p["ats"], **kw)
    M.mhc_fp8_gemm(p["aq"], p["aqs"], p["w2"], p["s2"], p["off"], p["ys"], **kw)
    M.mhc_fp8_quant(p["dys"], p["gq"], p["gqs"], p["gt"], p["gts"], **kw)
    M.mhc_fp8_gemm(p["gq"], p["gqs"], p["w2t"], p["s2t"], p["off"], p["da"], **kw)
    M.mhc_fp8_wgrad(p["gt"], p["gts"], p["at"], p["ats"], p["off"], p["dw2"], **kw)
    M.mhc_fp8_swiglu_bwd(p["da"], p["h"], None, p["hq"], p["hqs"], p["ht"], p["hts"], **kw)
    M.mhc_fp8_gemm(p["hq"], p["hqs"], p["w1t"], p["s1t"], p["off"], p["dxs"], **kw)
    M.mhc_fp8_wgrad(p["ht"], p["hts"], p["xt"], p["xts"], p["off"], p["dw1"], **kw)


def moe_tensors(M, counts, C, F, seed):
    E, off = len(counts), F8.segments(counts, 128)
    R = int(off[-1]) + 128
    p = {"off": off.cuda()}
    for n in ("xs", "dys"):
        t = torch.zeros(R, C)
        for lo, c in zip(off.tolist(), counts):
            t[lo:lo + c] = rows(c, C, seed + lo)
        p[n] = t.bfloat16().cuda()
    for n, a, b in (("1", 2 * F, C), ("2", C, F)):
        w = (rows(E * a, b, seed + 7).reshape(E, a, b) * b ** -0.5).bfloat16().cuda()
        p["w" + n], p["s" + n] = full(E, a, b, dtype=E4M3), full(E, blocks(b), blocks(a))
        p["w" + n + "t"], p["s" + n + "t"] = full(E, b, a, dtype=E4M3), full(E, blocks(a), blocks(b))
        M.mhc_fp8_quant(w, p["w" + n], p["s" + n], p["w" + n + "t"], p["s" + n + "t"], tiles=True)
    for n, c, fmt in (("x", C, E4M3), ("a", F, E4M3), ("g", C, E5M2), ("h", 2 * F, E5M2)):
        p[n + "q"], p[n + "qs"] = full(R, c, dtype=fmt), full(blocks(c), R)
        p[n + "t"], p[n + "ts"] = full(c, R, dtype=fmt), full(blocks(R), c)
    for n, c in (("h", 2 * F), ("ys", C), ("da", F), ("dxs", C)):
        p[n] = full(R, c, dtype=torch.bfloat16)
    p["dw1"], p["dw2"] = full(E, 2 * F, C), full(E, C, F)
    return p


def check_step(p, C, F):
    """Each step against 64 bits of what it was given."""
    off, cpu = p["off"].cpu(), {n: t.cpu() for n, t in p.items()}
    for a, w, s, out, K in (("xq", "w1", "s1", "h", C), ("aq", "w2", "s2", "ys", F),
                            ("gq", "w2t", "s2t", "da", C), ("hq", "w1t", "s1t", "dxs", 2 * F)):
        check(cpu[out], *gemm_ref(cpu[a], cpu[a + "s"], cpu[w], cpu[s], off), F8.product_ops(K), out)
    for g, a, out in (("gt", "at", "dw2"), ("ht", "xt", "dw1")):
        check(cpu[out], *wgrad_ref(cpu[g], cpu[g + "s"], cpu[a], cpu[a + "s"], off),
              F8.product_ops(1024), out)
    for src, n in (("xs", "x"), ("dys", "g")):
        fmt = cpu[n + "q"].dtype
        for got, ref in ((n + "q", F8.quant_rows(cpu[src].float(), fmt)),
                         (n + "t", F8.quant_rows(cpu[src].float().t().contiguous(), fmt))):
            assert torch.equal(bits(cpu[got]), bits(ref[0])) and torch.equal(cpu[got + "s"], ref[1])
    a, err = F8.swiglu(np64(cpu["h"]))
    F8.check_quantised(cpu["aq"], cpu["aqs"], a, err, "aq")
    F8.check_quantised(cpu["at"], cpu["ats"], a.T.copy(), err.T.copy(), "at")
    d, err = F8.swiglu_grad(np64(cpu["da"]), np64(cpu["h"]))
    F8.check_quantised(cpu["hq"], cpu["hqs"], d, err, "hq")
    F8.check_quantised(cpu["ht"], cpu["hts"], d.T.copy(), err.T.copy(), "ht")


def test_training_step_together(M):
    C, F = 272, 144
    p = moe_tensors(M, [130, 0, 5, 300], C, F, 31)
    moe_step(M, p)
    torch.cuda.synchronize()
    check_step(p, C, F)


def test_training_step_captured_and_on_another_stream(M):
    C, F = 144, 80
    p = moe_tensors(M, [130, 40], C, F, 12)
    moe_step(M, p)
    torch.cuda.synchronize()
    outs = ("h", "ys", "da", "dxs", "dw1", "dw2", "aq", "at", "hq", "ht", "aqs", "hts")
    want = {n: bits(p[n].view(torch.uint8)) for n in outs}
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe_step(M, p)
    for how in ("graph", "stream"):
        for n in outs:
            p[n].view(torch.uint8).fill_(255)
        torch.cuda.synchronize()
        if how == "graph":
            graph.replay()
            graph.replay()
        else:
            moe_step(M, p, stream=side)
        torch.cuda.synchronize()
        for n in outs:
            assert torch.equal(want[n], bits(p[n].view(torch.uint8))), (how, n)


def test_few_captured_and_back_to_back(M):
    """Two calls in a row on one workspace, and both replayed from a graph."""
    a = few_case(5, 160, 96, 6, 2, torch.bfloat16, True, 1)
    b = few_case(30, 160, 96, 6, 2, torch.bfloat16, True, 2)
    ws = M.workspace(M.OP_MOE_FEW_FWD, 30, 2, 256)
    fa, fb = few_run(M, a), few_run(M, b)
    ga, gb = ([None if t is None else t.cuda() for t in c] for c in (a, b))
    oa, ob = torch.empty_like(fa), torch.empty_like(fb)

    def calls():
        for (x, ids, w, w1, s1, w2, s2), o in ((ga, oa), (gb, ob)):
            M.mhc_moe_few_fwd(x, ids, w, w1, w2, o, ws, s1, s2)

    calls()
    torch.cuda.synchronize()
    assert torch.equal(oa, fa) and torch.equal(ob, fb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        oa.zero_()
        ob.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, fa) and torch.equal(ob, fb)


# ---- offsets past 32 bits, calls side by side --------------------------------

def random_e4m3(*shape):
    """Finite values of every sign and exponent, made on the device."""
    v = torch.empty(*shape, dtype=torch.uint8, device="cuda").random_(0, 0x7e)
    return v.view(E4M3)


def test_weights_past_32_bits(M):
    """The last of the experts stands past 2^32 bytes; it gives what it gives as the last of three
    (the few tokens' sums go by the number of slots and experts, so as many segments either way:
    min(experts, slots) = 3)."""
    E, F, C = 40, 4096, 16384
    w1, w2 = random_e4m3(E, 2 * F, C), random_e4m3(E, C, F)
    s1 = torch.rand(E, blocks(C), blocks(2 * F), device="cuda") * C ** -0.5
    s2 = torch.rand(E, blocks(F), blocks(C), device="cuda") * F ** -0.5
    x = rows(3, C, 1, torch.bfloat16).cuda() * 2.0 ** -6
    last = [t[-3:].clone() for t in (w1, s1, w2, s2)]
    ids = torch.full((3, 1), E - 1, dtype=I32, device="cuda")
    w = torch.ones(3, 1, device="cuda")
    out, one = full(3, C, dtype=torch.bfloat16), full(3, C, dtype=torch.bfloat16)
    ws = M.workspace(M.OP_MOE_FEW_FWD, 3, 1, C + F)
    M.mhc_moe_few_fwd(x, ids, w, w1, w2, out, ws, s1, s2)
    M.mhc_moe_few_fwd(x, torch.full_like(ids, 2), w, last[0], last[2], one, ws, last[1], last[3])
    assert torch.equal(out, one) and out.float().abs().max() > 0 and out.isfinite().all()
    xq, xs = full(3, C, dtype=E4M3), full(blocks(C), 3)
    M.mhc_fp8_quant(x, xq, xs)
    off = torch.tensor([0] * E + [3], dtype=I32, device="cuda")
    h, alone = full(3, 2 * F), full(3, 2 * F)
    M.mhc_fp8_gemm(xq, xs, w1, s1, off, h)
    M.mhc_fp8_gemm(xq, xs, last[0][2:], last[1][2:].clone(), None, alone)
    assert torch.equal(h, alone) and h.abs().max() > 0 and h.isfinite().all()


def test_rows_past_32_bits(M):
    """Quantised along both; the last rows and columns of 2^32 elements and more."""
    R, C = 262272, 16400
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_()
    q, s, qt, st = outputs(0, R, C, E4M3, False, "qt")
    M.mhc_fp8_quant(x, q, s, qt, st)
    tail = x[-128:].clone()
    tq, ts, tqt, tst = outputs(0, 128, C, E4M3, False, "qt")
    M.mhc_fp8_quant(tail, tq, ts, tqt, tst)
    assert torch.equal(bits(q[-128:]), bits(tq)) and torch.equal(s[:, -128:], ts)
    assert torch.equal(bits(qt[:, -128:]), bits(tqt)) and torch.equal(st[-1:], tst)


def test_calls_side_by_side(M):
    """Two streams, each with its own layer, products and workspace."""
    cases = [few_case(T, 272, 144, 12, 3, torch.bfloat16, eight, T) for T, eight in ((20, True), (64, False))]
    want = [few_run(M, c) for c in cases]
    gemms = [gemm_case([700, 130], 8, 1040, 400, E4M3, E4M3, n) for n in (5, 6)]
    gemms = [[t.cuda() for t in g[:5]] + [g[5]] for g in gemms]
    outs = [full(g[5], 1040) for g in gemms]
    for g, o in zip(gemms, outs):
        M.mhc_fp8_gemm(*g[:5], o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [[None if t is None else t.cuda() for t in c] for c in cases]
    ws = [M.workspace(M.OP_MOE_FEW_FWD, c[0].shape[0], 3, 272 + 144) for c in cases]
    got = [[full(*w.shape, dtype=w.dtype) for _ in range(8)] for w in want]
    prod = [[torch.empty_like(o) for _ in range(8)] for o in outs]
    torch.cuda.synchronize()
    for k in range(8):
        for n, st in enumerate(streams):
            x, ids, w, w1, s1, w2, s2 = dev[n]
            M.mhc_moe_few_fwd(x, ids, w, w1, w2, got[n][k], ws[n], s1, s2, stream=st)
            M.mhc_fp8_gemm(*gemms[n][:5], prod[n][k], stream=st)
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(g, want[n]) for g in got[n])
        assert all(torch.equal(p, outs[n]) for p in prod[n])
