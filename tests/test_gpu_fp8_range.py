"""The 8-bit floating-point operators and the experts' layer for a few tokens at the ends of
their range."""
import math

import numpy as np
import pytest
import torch

from tests import _fp8 as F8
from tests._edges import U, check, np64
from tests._fp8 import E4M3, E5M2, blocks
from tests.test_gpu_fp8 import (I32, few_case, few_ref, few_run, full, gemm_case, wgrad_case,
                                wgrad_ref)

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    yield m
    assert m.mhc_device_error() == 0


# ---- the activation between the two products of the few tokens' layer ---------

def one_expert(gate, up, w2, x, dtype):
    """One token, one expert, w = 1; gate and up [F, C], w2 [C, F], x [C], all exact in dtype."""
    exact = x[None], torch.cat((gate, up))[None], w2[None]
    x, w1, w2 = (t.to(dtype) for t in exact)
    assert all(torch.equal(t.float(), e) for t, e in zip((x, w1, w2), exact))
    return x, torch.zeros(1, 1, dtype=I32), torch.ones(1, 1), w1, None, w2, None


def gate_of_64():
    """silu(64) is 64 to the last bit of fp32, so h = 64 up where x[0] = 1."""
    g = torch.zeros(16, 16)
    g[:, 0] = 64.0
    return g


@pytest.mark.parametrize("dtype", HALVES)
def test_activation_keeps_the_bits_of_fp32(M, dtype):
    """h[i] = 64 (1 + 85 2^-14 + i 2^-20), exact in fp32; f[i] = h[i] - h[0] = i 2^-14 without any
    rounding."""
    x, up, w2 = torch.zeros(16), torch.zeros(16, 16), torch.eye(16)
    x[0], x[1] = 1.0, 2.0 ** -10
    up[:, 0], up[:, 1], up[:, 2] = 1.0, torch.arange(16) * 2.0 ** -10, 85 / 16
    x[2] = 2.0 ** -10
    w2[:, 0] -= 1
    f = few_run(M, one_expert(gate_of_64(), up, w2, x, dtype))
    assert np64(f)[0].tolist() == [i * 2.0 ** -14 for i in range(16)]


def test_small_fp16_activation_keeps_its_bits(M):
    """h[i] = (1 + i / 256) 2^-24, which fp16 holds as its least number; times 2^12."""
    x, up = torch.zeros(16), torch.zeros(16, 16)
    x[0], x[1] = 1.0, 2.0 ** -14
    up[:, 1] = (256 + torch.arange(16)) * 2.0 ** -24
    f = few_run(M, one_expert(gate_of_64(), up, torch.eye(16) * 2.0 ** 12, x, torch.float16))
    assert np64(f)[0].tolist() == [(1 + i / 256) * 2.0 ** -12 for i in range(16)]


def test_large_fp16_activation_is_kept(M):
    """h = 320 * 320 is above fp16's largest number, f = 16 h / 64 is not."""
    x, w = torch.ones(16), torch.full((16, 16), 20.0)
    f = few_run(M, one_expert(w, w, torch.full((16, 16), 1 / 64), x, torch.float16))
    assert np64(f)[0].tolist() == [25600.0] * 16


@pytest.mark.parametrize("T,C,F,E,k", [(1, 144, 400, 4, 2), (9, 272, 80, 3, 2), (30, 48, 1040, 4, 4)])
@pytest.mark.parametrize("dtype", HALVES)
def test_activations_of_all_sizes(M, T, C, F, E, k, dtype):
    """Activations from 1e-7 to 1e6 beside one another in a row."""
    x, ids, w, w1, s1, w2, s2 = few_case(T, C, F, E, k, dtype, False, 7 * T + F)
    size = 10 ** (torch.rand(F, generator=torch.Generator().manual_seed(F)) * 13 - 7)
    w1, w2 = w1.float(), w2.float()
    w1[:, :F] *= 10
    w1[:, F:] *= size[:, None].clamp(1e-3, 1e3)
    w2 /= size.clamp(1e-3, 1e3)
    case = (x, ids, w, w1.to(dtype), None, w2.to(dtype), None)
    f = few_run(M, case)
    assert f.isfinite().all()
    F8.check_few(f, *few_ref(case))


@pytest.mark.parametrize("dtype", HALVES)
def test_infinite_activation_beside_finite_ones(M, dtype):
    """An infinity in h goes to f as itself, whatever stands beside it; a NaN as a NaN."""
    x = torch.ones(1, 16)
    w1 = torch.full((1, 32, 16), 20.0)
    w1[0, 0] = math.inf
    w2 = torch.zeros(1, 16, 16)
    w2[0, :, 1] = -1.0           # of 102400
    w2[0, :, 0] = 1.0            # of the infinity
    w2[0, 8:, 0] = -1.0
    w2[0, 15, 0] = 0.0
    case = (x.to(dtype), torch.zeros(1, 1, dtype=I32), torch.ones(1, 1), w1.to(dtype), None,
            w2.to(dtype), None)
    f = np64(few_run(M, case))[0]
    assert f[:8].tolist() == [math.inf] * 8 and f[8:15].tolist() == [-math.inf] * 7
    assert math.isnan(f[15])


# ---- long sums ------------------------------------------------------------------

def thirds(s, dtype):
    """fp32 values as three of dtype, which hold all 24 bits."""
    out = []
    for _ in range(3):
        out.append(s.to(dtype))
        s = s - out[-1].float()
    assert not s.any()
    return torch.stack(out, -1)


def long_sum_error(M, which, K, n, dtype):
    """Of n sums of K positive products in the first (which = 1) or the second product: their
    relative errors, found as the difference of two experts: the second one's sum is three terms,
    the first one's rounded to fp32, which is exact; 64 of a gate of 64 is exact, too."""
    g = torch.Generator().manual_seed(K + n)
    C, F = (K, n) if which == 1 else (n, K)
    x, w1, w2 = torch.ones(1, C), torch.zeros(2, 2 * F, C), torch.zeros(2, C, F)
    w1[:, :F, 0] = 64.0
    if which == 1:
        x[0, 4:] = 1 + torch.rand(C - 4, generator=g)
        x = x.to(dtype).float()
        w1[0, F:] = (0.5 + torch.rand(F, C, generator=g)).to(dtype)
        s = w1[0, F:].double() @ x[0].double()
        w1[1, F:, 1:4] = thirds(s.float(), dtype).float()
        w2[:, torch.arange(F), torch.arange(F)] = 1.0
    else:
        u = (0.5 + torch.rand(F, generator=g)).to(dtype)
        w1[0, F:, 0] = u
        w1[1, F:F + 3, 0] = 1.0
        w2[0] = (0.5 + torch.rand(C, F, generator=g)).to(dtype)
        s = w2[0].double() @ u.double()
        w2[1, :, :3] = thirds(s.float(), dtype).float()
    ids = torch.tensor([[0, 1]], dtype=I32)
    f = few_run(M, (x.to(dtype), ids, torch.tensor([[1.0, -1.0]]), w1.to(dtype), None, w2.to(dtype),
                    None))
    f = f[0, :n].cpu().double() / 64
    return (f - (s - s.float().double())) / s


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("dtype", HALVES)
def test_long_sums_are_rounded_to_nearest(M, which, dtype):
    """Sums of 16384 products are right on the average.  Within a piece of 64 a tensor core cuts
    what it adds to by 2^-23 of it at most, at most 8 times, while it grows to the piece's sum:
    4.5 2^-23 of that; the pieces are added with rounding to nearest, which has no bias: 256
    additions of a 16th of the sum at most, off by 2^-24 / sqrt(3) of it (rms), and the mean of
    256 sums by a 16th of that, six times which is less than 2^-24."""
    error = long_sum_error(M, which, 16384, 256, dtype)
    assert abs(error.mean().item()) <= 10 * U
    assert error.abs().max().item() <= (9 + 16 + 16) * U  # and none beyond what each addition may be


# ---- batch-invariant mode ------------------------------------------------------

@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("C,F,E,k", [(1024, 512, 64, 2), (272, 1040, 8, 2), (4096, 176, 60, 4)])
def test_batch_invariant_mode(M, C, F, E, k, eight):
    """With the mode on a token's result has the same bits in every batch."""
    x, ids, w, w1, s1, w2, s2 = few_case(100, C, F, E, k, torch.bfloat16, eight, C + F)
    w1, s1, w2, s2 = (None if t is None else t.cuda() for t in (w1, s1, w2, s2))
    M.mhc_set_batch_invariant(True)
    try:
        out = few_run(M, (x, ids, w, w1, s1, w2, s2))
        F8.check_few(out, *few_ref((x, ids, w) + tuple(None if t is None else t.cpu()
                                                       for t in (w1, s1, w2, s2))))
        for lo, n in ((0, 1), (99, 1), (40, 2), (13, 17), (50, 50)):
            one = few_run(M, (x[lo:lo + n], ids[lo:lo + n], w[lo:lo + n], w1, s1, w2, s2))
            assert torch.equal(one, out[lo:lo + n]), (lo, n)
    finally:
        M.mhc_set_batch_invariant(False)


# ---- scales far apart ----------------------------------------------------------

# exponents of the two operands' scales; whether the 8-bit values are the least ones
SCALES = {"product past the largest": (70, 58, True), "product below the least": (-75, -70, False),
          "first large": (112, -100, False), "first small": (-118, 100, True),
          "second large": (-100, 112, False), "second small": (100, -118, True)}


def eight_bits(g, least, *shape):
    if least:  # subnormal: up to 7 / 512
        return (torch.randint(-7, 8, shape, generator=g) * 2.0 ** -9).to(E4M3)
    return (torch.randint(-28, 29, shape, generator=g) * 16.0).to(E4M3)


def scales(g, e, *shape):
    return (1 + torch.rand(*shape, generator=g)) * 2.0 ** e


def check_scaled(out, ref, mag, K, what=""):
    """fp32: the operations' roundings, the result's own, and the least subnormal."""
    g = np64(out)
    assert np.all(np.isfinite(g)), what
    tol = (F8.product_ops(K) + 1) * U * mag + 2.0 ** -149
    assert np.all(np.abs(g - ref) <= tol), (what, np.max(np.abs(g - ref) / (mag + 2.0 ** -149)))


@pytest.mark.parametrize("R,N,K", [(130, 264, 272), (4000, 2824, 144)])
@pytest.mark.parametrize("kind", SCALES)
def test_gemm_of_scales_far_apart(M, R, N, K, kind):
    ea, eb, least = SCALES[kind]
    g = torch.Generator().manual_seed(R)
    a, b = eight_bits(g, least, R, K), eight_bits(g, least, 1, N, K)
    a[7] = 0  # of a row of zeros comes a row of zeros
    sa, sb = scales(g, ea, blocks(K), R), scales(g, eb, 1, blocks(K), blocks(N))
    sa[0, :5] = 1.5 * 2.0 ** -eb  # and some whose scales' product is near 1
    out = full(R, N)
    M.mhc_fp8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), None, out)
    av, bv = F8.values(a, sa), F8.values(b[0], sb[0])
    check_scaled(out, av @ bv.T, np.abs(av) @ np.abs(bv).T, K, kind)
    assert not out[7].any()


# ---- the same of the weights' gradient --------------------------------------------

@pytest.mark.parametrize("R,M_,N", [(272, 130, 264), (144, 4000, 2824)])
@pytest.mark.parametrize("kind", SCALES)
def test_wgrad_of_scales_far_apart(M, R, M_, N, kind):
    """Of any size, but the first ones within [2^-94, 2^88]."""
    ea, eb, least = SCALES[kind]
    near = lambda e: min(max(e, -94), 87)  # noqa: E731
    g = torch.Generator().manual_seed(R)
    at, bt = eight_bits(g, least, M_, R), eight_bits(g, least, N, R)
    at[7], bt[9] = 0, 0
    sat, sbt = scales(g, near(ea), blocks(R), M_), scales(g, eb, blocks(R), N)
    sat[0, :5] = 1.5 * 2.0 ** near(-eb)
    out = full(1, M_, N)
    M.mhc_fp8_wgrad(at.cuda(), sat.cuda(), bt.cuda(), sbt.cuda(), None, out)
    av, bv = F8.values(at, sat), F8.values(bt, sbt)
    check_scaled(out[0], av @ bv.T, np.abs(av) @ np.abs(bv).T, R, kind)
    assert not out[0, 7].any() and not out[0, :, 9].any()


# ---- scales of the few tokens' layer ---------------------------------------------

def test_few_zeros_under_large_scales(M):
    """Weights of zeros give zeros, however large the scales' product is."""
    x = (torch.rand(3, 144) + 1).bfloat16() * 2.0 ** 80
    w1, s1 = torch.zeros(2, 64, 144).to(E4M3), torch.full((2, 2, 1), 2.0 ** 60)
    w2, s2 = torch.ones(2, 144, 32).to(E4M3), torch.ones(2, 1, 2)
    ids = torch.tensor([[0], [1], [1]], dtype=I32)
    assert not few_run(M, (x, ids, torch.ones(3, 1), w1, s1, w2, s2)).any()


def test_few_small_scales(M):
    """h is 2^-60, the second product's scales 2^-76: of their product fp32 holds four bits."""
    T, C, F = 3, 144, 128
    g = torch.Generator().manual_seed(3)
    x = (torch.rand(T, C, generator=g) + 1).bfloat16()
    w1 = torch.cat((torch.full((1, F, C), 0.5), torch.rand(1, F, C, generator=g) + 0.5), 1)
    s1 = torch.ones(1, blocks(C), 2)
    s1[:, :, 1] = 2.0 ** -73  # up
    w2, s2 = (torch.rand(1, C, F, generator=g) * 400 + 40).to(E4M3), scales(g, -76, 1, 1, blocks(C))
    case = (x, torch.zeros(T, 1, dtype=I32), torch.ones(T, 1), w1.to(E4M3), s1, w2, s2)
    f, err = few_ref(case)
    out = np64(few_run(M, case))
    assert np.abs(f).min() > 2.0 ** -125  # bf16's normal numbers
    assert np.all(np.abs(out - f) <= err + 2.0 ** -8 * (np.abs(f) + err))


def test_few_large_rows(M):
    """Rows of 2^121 under weights of 2^-125: a block's sum times the row's scale is past fp32."""
    T, C, F = 5, 272, 80
    g = torch.Generator().manual_seed(4)
    x = ((torch.rand(T, C, generator=g) + 1) * 2.0 ** 121).bfloat16()
    x[3] *= 2.0 ** -121
    w1 = torch.randint(-28, 29, (1, 2 * F, C), generator=g).float().to(E4M3)
    s1 = scales(g, -125, 1, blocks(C), 2)
    w2, s2 = eight_bits(g, False, 1, C, F), scales(g, -12, 1, 1, blocks(C))
    case = (x, torch.zeros(T, 1, dtype=I32), torch.ones(T, 1), w1, s1, w2, s2)
    f, err = few_ref(case)
    out = few_run(M, case)
    assert out.isfinite().all() and np.abs(f).max() > 1
    assert np.all(np.abs(np64(out) - f) <= err + 2.0 ** -8 * (np.abs(f) + err) + 2.0 ** -126)


# ---- segments' ends ---------------------------------------------------------------

@pytest.mark.parametrize("last,as_if", [(200, 128), (256, 256), (272, 272), (127, 0), (271, 256)])
def test_wgrad_of_a_last_end_off_the_blocks(M, last, as_if):
    """Any offset, the last one too, that is neither a multiple of 128 nor R is rounded down to
    one, and reported."""
    at, sat, bt, sbt, _ = wgrad_case([272], 40, 64, E4M3, E4M3, 5, 112)
    at, bt, sat, sbt = at[:, :272].clone(), bt[:, :272].clone(), sat[:3].clone(), sbt[:3].clone()
    sat = sat.nan_to_num(0.5)
    off = torch.tensor([0, last], dtype=I32)
    out = full(1, 40, 64)
    M.mhc_fp8_wgrad(*(t.cuda() for t in (at, sat, bt, sbt, off)), out)
    assert M.mhc_device_error() == (206 if last != as_if else 0)
    ref, mag = wgrad_ref(at, sat, bt, sbt, torch.tensor([0, as_if]))
    check(out, ref, mag, F8.product_ops(272))


# ---- rows of no segment -----------------------------------------------------------

def test_gemm_rows_behind_a_segment_are_not_used(M):
    """Rows of no segment may hold anything: an infinity and a NaN among the values and scales."""
    a, sa, b, sb, off, R = gemm_case([100, 60], 1, 64, 144, E5M2, E4M3, 3, 96)
    want, out = full(R, 64), full(R, 64)
    M.mhc_fp8_gemm(*(t.cuda() for t in (a, sa, b, sb, off)), want)
    raw = a.view(torch.uint8)
    raw[160:] = torch.tensor([0x7c, 0x7f, 0xfc, 0x7b], dtype=torch.uint8).repeat(36)
    sa[:, 160::2], sa[:, 161::2] = math.inf, 0.0
    M.mhc_fp8_gemm(*(t.cuda() for t in (a, sa, b, sb, off)), out)
    assert torch.equal(out, want) and not out[160:].any() and out.isfinite().all()


# ---- offsets past 32 bits ---------------------------------------------------------

def random_bits(*shape, small=False):
    """Finite e4m3 values of every sign and exponent, or such up to 2, made on the device."""
    v = torch.empty(*shape, dtype=torch.uint8, device="cuda").random_(0, 0x40 if small else 0x7e)
    return v.view(E4M3)


def test_wgrad_past_32_bits(M):
    """The results of the last of 17 segments stand past 2^32 elements."""
    G, M_, N = 17, 16384, 16392
    R = 128 * G
    at, bt = random_bits(M_, R), random_bits(N, R)
    sat = torch.rand(G, M_, device="cuda") + 0.5
    sbt = torch.rand(G, N, device="cuda") + 0.5
    off = torch.arange(G + 1, dtype=I32, device="cuda") * 128
    out = torch.full((G, M_, N), math.nan, dtype=torch.bfloat16, device="cuda")
    M.mhc_fp8_wgrad(at, sat, bt, sbt, off, out)
    for e in (0, G - 1):
        rows_ = slice(128 * e, 128 * e + 128)
        one = torch.full((1, M_, N), math.nan, dtype=torch.bfloat16, device="cuda")
        M.mhc_fp8_wgrad(at[:, rows_].contiguous(), sat[e:e + 1], bt[:, rows_].contiguous(),
                        sbt[e:e + 1], None, one)
        assert torch.equal(out[e], one[0]) and one.isfinite().all() and one.any()


def test_gemm_rows_past_32_bits(M):
    """R N past 2^32: the last segment ends inside a tile and a box, rows of no segment follow."""
    N, K = 16392, 144
    R = 262272 + 99
    end = R - 70
    a, b = random_bits(R, K), random_bits(2, N, K, small=True)
    sa = torch.rand(blocks(K), R, device="cuda") + 0.5
    sb = torch.rand(2, blocks(K), blocks(N), device="cuda") + 0.5
    off = torch.tensor([0, 262000, end], dtype=I32, device="cuda")
    out = torch.full((R, N), math.nan, dtype=torch.bfloat16, device="cuda")
    M.mhc_fp8_gemm(a, sa, b, sb, off, out)
    lo = end - 130
    one = torch.full((130, N), math.nan, dtype=torch.bfloat16, device="cuda")
    M.mhc_fp8_gemm(a[lo:end], sa[:, lo:end].contiguous(), b[1:], sb[1:].clone(), None, one)
    assert torch.equal(out[lo:end], one) and one.isfinite().all() and one.any()
    assert not out[end:].any()
    assert not out[:end].isnan().any(1).any()


@pytest.mark.parametrize("way", ["fwd", "bwd"])
def test_swiglu_past_32_bits(M, way):
    """R 2F past 2^32: the last rows, and the last columns of the transposed copy."""
    R, F = 262272, 8208
    h = torch.empty(R, 2 * F, dtype=torch.bfloat16, device="cuda").normal_()
    da = torch.empty(R, F, dtype=torch.bfloat16, device="cuda").normal_() if way == "bwd" else None
    C = F if way == "fwd" else 2 * F

    def run(h, da):
        n = h.shape[0]
        y = torch.full((n, C), math.nan, dtype=torch.bfloat16, device="cuda")
        q, qt = (torch.full(s, 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
                 for s in ((n, C), (C, n)))
        s, st = full(blocks(C), n), full(blocks(n), C)
        if way == "fwd":
            M.mhc_fp8_swiglu_fwd(h, y, q, s, qt, st)
        else:
            M.mhc_fp8_swiglu_bwd(da, h, y, q, s, qt, st)
        return y, q.view(torch.uint8), s, qt.view(torch.uint8), st

    y, q, s, qt, st = run(h, da)
    ty, tq, ts, tqt, tst = run(h[-128:].clone(), da[-128:].clone() if way == "bwd" else None)
    assert torch.equal(y[-128:], ty) and torch.equal(q[-128:], tq) and torch.equal(s[:, -128:], ts)
    assert torch.equal(qt[:, -128:], tqt) and torch.equal(st[-1:], tst)
    assert ty.isfinite().all() and ty.any()


# ---- other tokens of a segment ----------------------------------------------------

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("eight", [False, True])
def test_few_bits_beside_a_token_out_of_range(M, dtype, eight):
    """A token that holds an infinity, a NaN or the type's largest number leaves the bits of the
    seven beside it as they are."""
    case = few_case(8, 1040, 2048, 1, 1, dtype, eight, 5, 0.0)
    out = few_run(M, case)
    for v in (math.inf, math.nan, torch.finfo(dtype).max):
        x = case[0].clone()
        x[5, 3] = v
        again = few_run(M, (x,) + case[1:])
        keep = torch.arange(8, device="cuda") != 5
        assert torch.equal(again[keep], out[keep]), v
