"""Refusals of the 8-bit floating-point operators: every bad argument is found
on the host, before a device is touched."""
import pytest
import torch

A = 0x10000  # a 16-byte-aligned fake device address; never dereferenced
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def M():
    from layers_proj_rms_gb300 import build as B
    B.build()
    import layers_proj_rms_gb300 as m
    return m


@pytest.fixture(scope="module")
def L(M):
    return M.lib


def quant(L, x=A, dt=0, G=1, R=32, C=64, fmt=0, tiles=0, q=A, s=A, qt=A, st=A):
    return L.mhc_fp8_quant(x, dt, G, R, C, fmt, tiles, q, s, qt, st, None)


# (keyword arguments, status): 1 null, 2 shape, 3 alignment, 6 argument
@pytest.mark.parametrize("kw,status", [
    ({"dt": 3}, 6), ({"fmt": 2}, 6), ({"fmt": -1}, 6), ({"G": -1}, 2), ({"G": 65536}, 2),
    ({"R": -1}, 2), ({"R": 1 << 31}, 2), ({"C": 0}, 2), ({"C": 24}, 2), ({"R": 24}, 2),
    ({"R": 24, "qt": None}, 2), ({"C": (1 << 30) + 16}, 2),
    ({"R": (1 << 31) - 16, "C": 1 << 30}, 2), ({"x": None}, 1), ({"s": None}, 1), ({"q": None}, 1),
    ({"st": None}, 1), ({"x": A + 8}, 3), ({"q": A + 8}, 3), ({"st": A + 4}, 3),
    ({"q": None, "s": None, "qt": None, "st": None}, 1),
])
def test_quant_refuses(L, kw, status):
    assert quant(L, **kw) == status
    assert L.mhc_last_error()


def test_quant_accepts_nothing_to_do(L):
    none = {"x": None, "q": None, "s": None, "qt": None, "st": None}
    assert quant(L, R=0, **none) == 0 and quant(L, G=0, **none) == 0


def test_quant_accepts_without_gpu(L):
    assert quant(L) in (7, 8)
    assert quant(L, R=24, qt=None, st=None) in (7, 8)
    assert quant(L, q=None, s=None) in (7, 8)


def test_swiglu_refuses(L):
    f = lambda h=A, dt=0, R=32, F=64, fmt=0, a=None, q=A, s=A, qt=A, st=A: L.mhc_fp8_swiglu_fwd(  # noqa: E731
        h, dt, R, F, fmt, a, q, s, qt, st, None)
    assert f(F=24) == 2 and f(F=0) == 2 and f(R=-1) == 2 and f(R=24) == 2 and f(dt=9) == 6
    assert f(fmt=2) == 6 and f(h=None) == 1 and f(h=A + 2) == 3 and f(a=A + 8) == 3
    assert f(q=None) == 1 and f(q=None, s=None, qt=None, st=None) == 1
    assert f(R=0, h=None) == 0
    b = lambda da=A, h=A, R=32, F=64, dh=None, q=A, s=A, qt=None, st=None: L.mhc_fp8_swiglu_bwd(  # noqa: E731
        da, h, 0, R, F, 0, dh, q, s, qt, st, None)
    assert b(da=None) == 1 and b(h=None) == 1 and b(F=40) == 2 and b(da=A + 8) == 3
    assert b(st=A) == 1 and b(R=0, da=None) == 0


def gemm(L, a=A, fa=0, sa=A, b=A, fb=0, sb=A, off=A, G=4, R=64, N=64, K=64, dt=0, out=A):
    return L.mhc_fp8_gemm(a, fa, sa, b, fb, sb, off, G, R, N, K, dt, out, None)


@pytest.mark.parametrize("kw,status", [
    ({"fa": 2}, 6), ({"fb": -1}, 6), ({"dt": 3}, 6), ({"G": 0}, 2), ({"G": 1025}, 2), ({"R": -1}, 2),
    ({"R": 1 << 31}, 2), ({"N": 0}, 2), ({"N": 12}, 2), ({"K": 8}, 2), ({"K": 24}, 2), ({"K": 0}, 2),
    ({"R": (1 << 31) - 1, "N": (1 << 31) - 8}, 2), ({"off": None}, 1), ({"off": A + 2}, 3),
    ({"a": None}, 1), ({"sa": None}, 1), ({"b": None}, 1), ({"sb": None}, 1), ({"out": None}, 1),
    ({"a": A + 8}, 3), ({"b": A + 8}, 3), ({"out": A + 8}, 3),
])
def test_gemm_refuses(L, kw, status):
    assert gemm(L, **kw) == status
    assert L.mhc_last_error()


def test_gemm_accepts_nothing_to_do(L):
    assert gemm(L, R=0, a=None, out=None) == 0


def test_products_accept_without_gpu(L):
    assert gemm(L) in (7, 8) and gemm(L, off=None, G=1) in (7, 8)
    assert gemm(L, off=A + 4) in (7, 8)
    assert wgrad(L) in (7, 8) and wgrad(L, off=None, G=1, M=1) in (7, 8)
    assert wgrad(L, R=0, at=None) in (7, 8)  # zeros are written


def wgrad(L, at=A, fa=0, sa=A, bt=A, fb=0, sb=A, off=A, G=4, R=64, M=64, N=64, dt=2, out=A):
    return L.mhc_fp8_wgrad(at, fa, sa, bt, fb, sb, off, G, R, M, N, dt, out, None)


@pytest.mark.parametrize("kw,status", [
    ({"fa": 2}, 6), ({"fb": 2}, 6), ({"dt": -1}, 6), ({"G": 0}, 2), ({"G": 1025}, 2), ({"R": 24}, 2),
    ({"R": -16}, 2), ({"M": 0}, 2), ({"N": 20}, 2), ({"off": None}, 1), ({"at": None}, 1),
    ({"sb": None}, 1), ({"out": None}, 1), ({"bt": A + 8}, 3), ({"out": A + 4}, 3),
    ({"M": (1 << 31) - 128, "N": 1 << 30, "G": 1024}, 2),
])
def test_wgrad_refuses(L, kw, status):
    assert wgrad(L, **kw) == status
    assert L.mhc_last_error()


@pytest.mark.parametrize("R", [(1 << 31) - 127, (1 << 31) - 112, (1 << 31) - 16, (1 << 31) - 1])
def test_products_refuse_rows_that_tiles_count_past_32_bits(L, R):
    assert gemm(L, R=R, N=8, K=16, G=1) == 2
    assert wgrad(L, R=(1 << 31) - 16, M=8, N=8, G=1) == 2
    for f in gemm, wgrad:
        assert f(L, R=(1 << 31) - 128, N=8, G=1) in (7, 8)


def few(L, x=A, dt=0, ids=A, w=A, w1=A, s1=None, w2=A, s2=None, T=4, k=2, E=8, C=64, F=32, f=A, ws=A,
        nb=1 << 20):
    return L.mhc_moe_few_fwd(x, dt, ids, w, w1, s1, w2, s2, T, k, E, C, F, f, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    ({"dt": 2}, 6), ({"dt": -1}, 6), ({"T": -1}, 2), ({"T": 129}, 2), ({"k": 0}, 2), ({"k": 33}, 2),
    ({"E": 0}, 2), ({"E": 1025}, 2), ({"C": 24}, 2), ({"C": 0}, 2), ({"C": 16400}, 2), ({"F": 8}, 2),
    ({"F": 16400}, 2), ({"s1": A}, 1), ({"s2": A}, 1), ({"x": None}, 1), ({"ids": None}, 1),
    ({"w": None}, 1), ({"w1": None}, 1), ({"w2": None}, 1), ({"f": None}, 1), ({"ws": None}, 1),
    ({"w1": A + 8}, 3), ({"ws": A + 16}, 3), ({"nb": 16}, 5),
])
def test_few_refuses(L, kw, status):
    assert few(L, **kw) == status
    assert L.mhc_last_error()


def test_few_workspace(M, L):
    ws = M.mhc_workspace_bytes
    need = ws(M.OP_MOE_FEW_FWD, 4, 2, 96)
    assert need >= 4 * 2 * 96 * 4 and need % 256 == 0
    assert few(L, nb=need - 1) == 5 and few(L, T=0, x=None, ws=None, nb=0) == 0
    assert ws(M.OP_MOE_FEW_FWD, 129, 2, 96) == 0 and ws(M.OP_MOE_FEW_FWD, 4, 33, 96) == 0
    assert ws(M.OP_MOE_FEW_FWD, 4, 2, 97) == 0 and ws(M.OP_MOE_FEW_FWD, -1, 2, 96) == 0


def test_few_accepts_without_gpu(M, L):
    need = M.mhc_workspace_bytes(M.OP_MOE_FEW_FWD, 4, 2, 96)
    assert few(L, nb=need) in (7, 8) and few(L, nb=need, s1=A, s2=A, dt=1) in (7, 8)


def test_binding_names_what_is_wrong(M):
    """Each refused by name before a device is looked at (no tensor here is on one)."""
    meta = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    x, q, s = meta(32, 160), meta(32, 160, dt=E4), meta(2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        M.mhc_fp8_quant(x, q, s)
    with pytest.raises(TypeError, match="q: dtype torch.uint8, expected float8"):
        M.mhc_fp8_quant(torch.empty(0, 160), torch.empty(0, 160, dtype=torch.uint8), s)
    with pytest.raises(ValueError, match=r"x must have 2 dimensions"):
        M.mhc_fp8_quant(meta(160), q, s)
    with pytest.raises(ValueError, match="x must be contiguous"):
        M.mhc_fp8_quant(meta(160, 32).t(), q, s)
    e = torch.empty(0, 160, dtype=E4)
    none = torch.empty(0, 160)
    with pytest.raises(TypeError, match="s must be a torch.Tensor"):
        M.mhc_fp8_quant(none, e)
    with pytest.raises(ValueError, match=r"s: shape .*expected \(2, 0\)"):
        M.mhc_fp8_quant(none, e, torch.empty(1, 0))
    with pytest.raises(ValueError, match=r"s: shape .*expected \(2, 0\)"):
        M.mhc_fp8_quant(none, e, torch.empty(0, 2), tiles=True)
    with pytest.raises(TypeError, match="qt: dtype torch.float8_e5m2, expected torch.float8_e4m3fn"):
        M.mhc_fp8_quant(none, e, torch.empty(2, 0), torch.empty(160, 0, dtype=E5), torch.empty(0, 160))
    M.mhc_fp8_quant(none, e, torch.empty(2, 0))  # no rows
    with pytest.raises(ValueError, match="halves"):
        M.mhc_fp8_swiglu_fwd(torch.empty(0, 33))
    with pytest.raises(ValueError, match=r"q: shape .*expected \(0, 320\)"):
        M.mhc_fp8_swiglu_bwd(none, torch.empty(0, 320), None, e, torch.empty(3, 0))
    a, b = torch.empty(0, 160, dtype=E4), meta(2, 24, 160, dt=E4)
    with pytest.raises(ValueError, match="b must have 3 dimensions"):
        M.mhc_fp8_gemm(a, None, meta(24, 160, dt=E4), None, None, torch.empty(0, 24))
    with pytest.raises(ValueError, match="CUDA"):
        M.mhc_fp8_gemm(a, torch.empty(2, 0), b, meta(2, 2, 1), None, torch.empty(0, 24))
    with pytest.raises(TypeError, match="a: dtype torch.float32"):
        M.mhc_fp8_gemm(a.float(), None, b, None, None, torch.empty(0, 24))
    with pytest.raises(ValueError, match=r"bt: shape .*expected \(24, 0\)"):
        M.mhc_fp8_wgrad(torch.empty(16, 0, dtype=E4), None, meta(24, 16, dt=E4), None, None,
                        meta(1, 16, 24))
    xb = torch.empty(0, 64, dtype=torch.bfloat16)
    ids, w = torch.empty(0, 2, dtype=torch.int32), torch.empty(0, 2)
    with pytest.raises(TypeError, match="w1: dtype torch.bfloat16, expected torch.float8_e4m3fn"):
        M.mhc_moe_few_fwd(xb, ids, w, meta(4, 64, 64, dt=torch.bfloat16),
                          meta(4, 64, 32, dt=torch.bfloat16), xb, None, meta(4, 1, 1), meta(4, 1, 1))
    with pytest.raises(ValueError, match=r"w1: shape .*expected \(4, 64, 64\)"):
        M.mhc_moe_few_fwd(xb, ids, w, meta(4, 32, 64, dt=torch.bfloat16),
                          meta(4, 64, 32, dt=torch.bfloat16), xb, None)
