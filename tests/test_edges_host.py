"""Refusals of the sub-layer edge operators (q/k norm + rotation, router, sort,
dispatch, combine): every bad argument is found on the host, before a device
is touched."""
import pytest
import torch

A = 0x10000  # a 16-byte-aligned fake device address; never dereferenced
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    from layers_proj_rms_gb300 import build as B
    B.build()
    import layers_proj_rms_gb300 as m
    return m


def fwd(L, q=A, k=A, dtype=0, strides=None, gq=A, gk=A, cos=A, sin=A, pos=A, T=4, Hq=2, Hk=1,
        D=64, R=64, P=16, inter=0, eps=EPS, qo=2 * A, ko=3 * A):
    st = (L.c_strides * len(strides))(*strides) if strides else None
    return L.mhc_qk_norm_rope_fwd(q, k, dtype, st, gq, gk, cos, sin, pos, T, Hq, Hk, D, R, P,
                                  inter, eps, qo, ko, None)


@pytest.fixture(scope="module")
def L(M):
    import ctypes
    M.lib.c_strides = ctypes.c_int64
    return M.lib


# (keyword arguments, status): 1 null, 2 shape, 3 alignment, 6 argument
@pytest.mark.parametrize("kw,status", [
    ({"dtype": 3}, 6), ({"dtype": -1}, 6), ({"T": -1}, 2), ({"Hq": -1}, 2), ({"D": 0}, 2),
    ({"D": 513}, 2), ({"R": 65}, 2), ({"R": 33}, 2), ({"R": -2}, 2), ({"P": -1}, 2), ({"T": 1 << 31}, 2), ({"P": 1 << 31}, 2),
    ({"eps": float("nan")}, 6), ({"eps": -1.0}, 6), ({"q": None}, 1), ({"ko": None}, 1),
    ({"cos": None}, 1), ({"sin": None}, 1), ({"q": A + 1}, 3), ({"dtype": 2, "k": A + 2}, 3),
    ({"gq": A + 4}, 3), ({"pos": A + 2}, 3), ({"pos": None, "T": 17}, 2),
    # output heads that overlap: by token, by head; a negative stride
    ({"strides": [128, 64, 64, 64, 127, 64, 64, 64]}, 2),
    ({"strides": [128, 64, 64, 64, 128, 63, 64, 64]}, 2),
    ({"strides": [-128, 64, 64, 64, 128, 64, 64, 64]}, 2),
    # in place with other strides
    ({"qo": A, "strides": [256, 64, 64, 64, 128, 64, 64, 64]}, 2),
])
def test_qk_forward_refuses(L, kw, status):
    assert fwd(L, **kw) == status
    assert L.mhc_last_error()


def test_qk_forward_accepts(L):
    """What passes the checks reaches the device check (or is a no-op)."""
    assert fwd(L, T=0, q=None, k=None, qo=None, ko=None, cos=None, sin=None, pos=None) == 0
    assert fwd(L, Hq=0, Hk=0, q=None, k=None, qo=None, ko=None) == 0
    if torch.cuda.is_available():
        return  # the addresses are not real
    ok = (7, 8)
    assert fwd(L) in ok
    assert fwd(L, R=0, cos=None, sin=None, pos=None, P=0) in ok
    assert fwd(L, q=A + 2, T=3) in ok                    # element alignment is enough
    assert fwd(L, Hk=0, k=None, ko=None) in ok
    assert fwd(L, gq=None, gk=None, pos=None) in ok
    assert fwd(L, strides=[0, 0, 64, 64, 64, 256, 64, 64]) in ok  # head-major out, broadcast in
    assert fwd(L, qo=A, ko=A + 4096) in ok               # in place


def bwd(L, up=A, q=A, dq=2 * A, dgq=A, dgk=A, ws=A, nb=1 << 20, T=4, Hq=2, Hk=1, D=64, R=64):
    return L.mhc_qk_norm_rope_bwd(up, 5 * A, q, 6 * A, 0, None, A, A, A, A, A, T, Hq, Hk, D, R,
                                  16, 0, EPS, dq, 7 * A, dgq, dgk, ws, nb, None)


def test_qk_backward_refuses(M, L):
    need = M.mhc_workspace_bytes(M.OP_QK_NORM_ROPE_BWD, 4, 3, 64)
    assert need > 0 and need % 256 == 0
    assert bwd(L, up=None) == 1 and bwd(L, dq=None) == 1
    assert bwd(L, nb=need - 1) == 5 and bwd(L, ws=None) == 1 and bwd(L, ws=A + 16) == 3
    assert bwd(L, R=7) == 2 and bwd(L, dgq=A + 4) == 3
    if not torch.cuda.is_available():
        assert bwd(L, nb=need) in (7, 8)
        assert bwd(L, dgq=None, dgk=None, ws=None, nb=0) in (7, 8)  # frozen gammas: no workspace
    ws = M.mhc_workspace_bytes
    assert ws(13, 0, 3, 64) == 0 and ws(13, 4, 0, 64) == 0 and ws(13, 4, 3, 513) == 0
    assert ws(13, 1 << 20, 40, 128) == ws(13, 1 << 24, 40, 128) > 0  # bounded
    assert ws(13, 1 << 20, 40, 33) > 0                               # any head size


def test_router_refuses(L):
    f = lambda T=4, E=8, k=2, dt=0, sc=0, scale=1.0, x=A, ids=A, w=A: L.mhc_moe_router_fwd(  # noqa: E731
        x, dt, T, E, k, sc, 1, scale, ids, w, None)
    assert f(T=-1) == 2 and f(E=0) == 2 and f(E=1025) == 2 and f(k=0) == 2 and f(k=9) == 2
    assert f(E=64, k=33) == 2 and f(dt=3) == 6 and f(sc=2) == 6 and f(scale=float("inf")) == 6
    assert f(x=None) == 1 and f(ids=None) == 1 and f(w=A + 4) == 3
    assert f(T=0, x=None, ids=None, w=None) == 0
    b = lambda dw=A, x=A, ids=A, dl=A, T=4, k=2: L.mhc_moe_router_bwd(  # noqa: E731
        dw, x, 0, ids, T, 8, k, 0, 1, 1.0, dl, None)
    assert b(dw=None) == 1 and b(ids=None) == 1 and b(dl=A + 8) == 3 and b(k=9) == 2
    assert b(T=0, dw=None) == 0


def test_sort_refuses(M, L):
    rows = M.mhc_moe_rows(10, 2, 4, 8)
    assert rows == 20 + 4 * 7 and M.mhc_moe_rows(1, 2, 4, 8) == 2 + 2 * 7
    assert M.mhc_moe_rows(0, 2, 4, 8) == 0
    for bad in ((-1, 2, 4, 8), (1, 0, 4, 8), (1, 33, 4, 8), (1, 2, 0, 8), (1, 2, 1025, 8),
                (1, 2, 4, 0), (1, 2, 4, 65537)):
        assert M.mhc_moe_rows(*bad) == -1
    f = lambda T=10, k=2, E=4, al=8, R=rows, ids=A, c=A, o=A, ro=A, so=A: L.mhc_moe_sort(  # noqa: E731
        ids, T, k, E, al, R, c, o, ro, so, None)
    assert f(R=rows - 1) == 2 and f(T=-1) == 2 and f(k=33) == 2 and f(E=0) == 2 and f(al=0) == 2
    assert f(T=1 << 30, k=2, R=(1 << 31) - 1) == 2 and f(R=1 << 31) == 2
    assert f(ids=None) == 1 and f(c=None) == 1 and f(ro=None) == 1 and f(so=None) == 1
    assert f(o=A + 4) == 3


def test_rows_refuse(L):
    d = lambda T=4, k=2, R=16, C=64, dt=0, x=A, ro=A, so=A, xs=A: L.mhc_moe_dispatch_fwd(  # noqa: E731
        x, dt, ro, so, T, k, R, C, xs, None)
    assert d(C=60) == 2 and d(C=0) == 2 and d(k=0) == 2 and d(R=-1) == 2 and d(dt=5) == 6
    assert d(x=None) == 1 and d(so=None) == 1 and d(xs=A + 8) == 3
    assert d(R=0, x=None, ro=None, so=None, xs=None) == 0
    b = lambda T=4, R=16, g=A, dx=A: L.mhc_moe_dispatch_bwd(g, 0, A, T, 2, R, 64, dx, None)  # noqa: E731
    assert b(g=None) == 1 and b(dx=None) == 1 and b(T=1 << 31) == 2 and b(T=0, g=None) == 0
    c = lambda T=4, R=16, C=64, ys=A, w=A, f=A: L.mhc_moe_combine_fwd(  # noqa: E731
        ys, 0, w, A, T, 2, R, C, f, None)
    assert c(ys=None) == 1 and c(w=A + 4) == 3 and c(f=None) == 1 and c(C=12) == 2
    assert c(T=0, ys=None, f=None) == 0
    g = lambda T=4, R=16, df=A, ys=A, dys=A, dw=A, so=A: L.mhc_moe_combine_bwd(  # noqa: E731
        df, ys, 0, A, A, so, T, 2, R, 64, dys, dw, None)
    assert g(df=None) == 1 and g(ys=None) == 1 and g(dys=None) == 1 and g(so=None) == 1
    assert g(dw=A + 4) == 3 and g(T=0, R=0, df=None, ys=None, dys=None) == 0


def test_binding_refuses(M):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        M.mhc_qk_norm_rope_fwd(x, x, None, None, None, None, None, EPS, x, x)
    with pytest.raises(TypeError, match="float64|dtype"):
        M.mhc_qk_norm_rope_fwd(x.double(), x.double(), None, None, None, None, None, EPS,
                               x.double(), x.double())
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        M.mhc_qk_norm_rope_fwd(x[0], None, None, None, None, None, None, EPS, x[0], None)
    with pytest.raises(ValueError, match="contiguous"):
        M.mhc_qk_norm_rope_fwd(x[..., ::2], None, None, None, None, None, None, EPS, x[..., ::2],
                               None)
    with pytest.raises(TypeError, match="dtype"):
        M.mhc_moe_dispatch_fwd(x[0].int(), x[0].int(), x[0].int(), x[0].int())


def test_binding_names_what_is_wrong(M):
    """Types, shapes, dimensions, missing tensors: each refused by name before a
    device is looked at (the tensors here are on the CPU)."""
    i32, bf = torch.int32, torch.bfloat16
    meta = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    ids, w, cnt, off = meta(4, 2, dt=i32), meta(4, 2), meta(5, dt=i32), meta(6, dt=i32)
    row, slot = meta(4, 2, dt=i32), meta(8, dt=i32)
    with pytest.raises(TypeError, match="ids must be a torch.Tensor"):
        M.mhc_moe_sort([[1]], 1, cnt, off, row, slot)
    with pytest.raises(TypeError, match="counts must be a torch.Tensor"):
        M.mhc_moe_sort(ids, 1, None, off, row, slot)
    with pytest.raises(ValueError, match="CUDA"):
        M.mhc_moe_sort(ids, 1, cnt, off, row, slot)
    with pytest.raises(TypeError, match="ids: dtype torch.int64, expected torch.int32"):
        M.mhc_moe_sort(ids.long(), 1, cnt, off, row, slot)
    with pytest.raises(ValueError, match="2 dimensions"):
        M.mhc_moe_sort(cnt, 1, cnt, off, row, slot)
    e = torch.empty(0, dtype=i32)
    with pytest.raises(ValueError, match=r"offsets: shape .*expected \(1,\)"):
        M.mhc_moe_sort(e.view(0, 2), 1, e, e, e.view(0, 2), e)
    logits = meta(4, 8)
    with pytest.raises(TypeError, match="logits: dtype torch.int32"):
        M.mhc_moe_router_fwd(logits.int(), 0, True, 1.0, ids, w)
    q = torch.empty(0, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="both None"):
        M.mhc_qk_norm_rope_fwd(None, None, None, None, None, None, None, EPS, None, None)
    with pytest.raises(TypeError, match="q_out must be a torch.Tensor"):
        M.mhc_qk_norm_rope_fwd(q, None, None, None, None, None, None, EPS, None, None)
    with pytest.raises(TypeError, match="q_out: dtype torch.float32, expected torch.bfloat16"):
        M.mhc_qk_norm_rope_fwd(q, None, None, None, None, None, None, EPS, q.float(), None)
    with pytest.raises(ValueError, match=r"q_out: shape .*expected \(0, 2, 64\)"):
        M.mhc_qk_norm_rope_fwd(q, None, None, None, None, None, None, EPS, q[:, :1], None)
    M.mhc_qk_norm_rope_fwd(q, None, None, None, None, None, None, EPS, q, None)  # no tokens
