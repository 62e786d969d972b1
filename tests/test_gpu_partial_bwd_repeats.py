"""The projection backward without the layer terms (the channel-sharded and the
standalone op, n = 4), called back to back: no wait in it may run out.  Its
epilogue used to wait for the du_hl part of a stage that it does not hold back;
a warp that came late missed that phase and waited for one that waited for it,
in about one of fifty calls at this size."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_partial_bwd_back_to_back():
    import layers_proj_rms_gb300 as M
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, n, Cs = 16384, 4, 2048
    O = n * n + 2 * n
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, n, Cs, generator=g, device="cuda").bfloat16()
    W = 0.02 * torch.randn(n * Cs, O, generator=g, device="cuda")
    du, coef = torch.randn(T, O, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    ws = M.workspace(M.OP_PROJ_RMS_PARTIAL_BWD, T, n, Cs)
    M.mhc_device_error()
    first = None
    for _ in range(8):
        for _ in range(100):
            M.mhc_proj_rms_partial_bwd(x, W, du, coef, dx, dW, ws)
        assert M.mhc_device_error() == 0
        if first is None:
            first = dx.clone(), dW.clone()
        assert torch.equal(dx, first[0]) and torch.equal(dW, first[1])
