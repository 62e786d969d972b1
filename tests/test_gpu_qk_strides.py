"""q/k norm + rotation of tokens in views whose strides are off 16 bytes: one
token, a few and all of them give the same bits."""
import pytest
import torch

from tests import _edges as O
from tests.test_gpu_qk import make, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def padded(t, extra):
    """The same tokens, `extra` elements between one and the next."""
    T, H, D = t.shape
    rows = torch.full((T, H * D + extra), 9.0, dtype=t.dtype, device="cuda")
    rows[:, :H * D] = t.reshape(T, H * D)
    return rows[:, :H * D].view(T, H, D)


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("extra", [1, 2, 4, 6, 8])
@pytest.mark.parametrize("Hq,Hk,D,R,inter", [(32, 8, 128, 128, False), (3, 1, 80, 20, True)])
def test_a_token_of_a_padded_view_does_not_depend_on_the_batch(M, Hq, Hk, D, R, inter, extra, dt):
    T = 11
    d = make(T, Hq, Hk, D, R, dt, seed=11)
    d.update({n: padded(d[n], extra) for n in ("q", "k", "dq", "dk")})
    dense = lambda d: tuple(torch.empty(d[n].shape, dtype=dt, device="cuda") for n in "qk")  # noqa: E731

    def both(d):
        q, k = run_fwd(M, d, inter, None, None, *dense(d))
        return (q, k) + run_bwd(M, d, inter, *dense(d))[:2]

    every = both(d)
    for a, b in [(t, t + 1) for t in range(T)] + [(0, 2), (5, 9)]:
        part = {n: (v[a:b] if n in ("q", "k", "dq", "dk", "pos") else v) for n, v in d.items()}
        assert part["q"].stride(0) == Hq * D + extra
        for x, y in zip(both(part), every):
            assert torch.equal(x, y[a:b])
    assert M.mhc_device_error() == 0
