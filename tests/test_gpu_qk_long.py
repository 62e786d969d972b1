"""q/k norm + rotation on long inputs of the head sizes that fill their lanes
(64, 128, 256), with more heads than a warp has lane groups: rotated whole and
in part, both pairings."""
import pytest
import torch

from tests import _edges as O
from tests.test_gpu_qk import EPS, make, run_bwd, run_fwd, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(701, 12, 2, 64, 64), (502, 17, 9, 64, 32),
                                         (1001, 9, 1, 128, 128), (613, 12, 5, 128, 96),
                                         (900, 8, 3, 256, 256), (1201, 7, 2, 256, 64)])
def test_forward_and_backward(M, T, Hq, Hk, D, R, inter, dt):
    assert T * (Hq + Hk) >= 152 * 64 and Hq > 32 * 16 // D
    d = make(T, Hq, Hk, D, R, dt, seed=12)
    got = run_fwd(M, d, inter)
    dq, dk, dgq, dgk = run_bwd(M, d, inter)
    for y, gy, gg, x, u, g, H in ((got[0], dq, dgq, "q", "dq", "gq", Hq),
                                  (got[1], dk, dgk, "k", "dk", "gk", Hk)):
        args = O.np64(d[x]), O.np64(d[g]), *table(d), R, inter, EPS
        # rho: the sum of D squares, its root; then gamma and the rotation
        O.check(y, *O.qk_fwd(*args), D / 2 + 12, x)
        # rho twice and the sum of D products; dgamma: the sum of T H products of them
        dx, dxm, dg, dgm = O.qk_bwd(O.np64(d[u]), *args)
        O.check(gy, dx, dxm, 2 * D + 20, "d" + x)
        O.check(gg, dg, dgm, T * H + D + 20, "dgamma " + x)
    # a few tokens of them, which the forms for short inputs take
    part = {n: (v[T // 2:T // 2 + 3] if n in ("q", "k", "dq", "dk", "pos") else v)
            for n, v in d.items()}
    few = run_fwd(M, part, inter) + run_bwd(M, part, inter)[:2]
    for a, b in zip(few, got + (dq, dk)):
        assert torch.equal(a, b[T // 2:T // 2 + 3])
    assert M.mhc_device_error() == 0
