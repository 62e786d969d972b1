"""Router gradient after slots of the choice were dropped (id -1): that of the
forward's weights over the whole choice, the dropped slots' dw being 0."""
import numpy as np
import pytest
import torch

from tests import _edges as O
from tests.test_gpu_moe import exp_ops, rng, route, route_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import layers_proj_rms_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def drop(ids, share, seed):
    """ids with about `share` of the slots dropped; which were kept."""
    keep = torch.rand(ids.shape, generator=rng(seed)).cuda() >= share
    return torch.where(keep, ids, -1).int().contiguous(), keep


@pytest.mark.parametrize("dt", O.DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 6, 3), (3, 1, 1), (40, 61, 4), (70, 8, 8), (9, 1024, 32),
                                   (20, 33, 32), (17, 256, 8)])
def test_dropped_slots_keep_their_share_of_the_sum(M, T, E, k, score, renorm, dt):
    g = rng(T * E)
    l = (2 * torch.randn(T, E, generator=g)).to(dt).cuda()
    ids, _ = route(M, l, k, score, renorm, 2.5)
    dw = torch.randn(T, k, generator=g).cuda()
    for share in (0.3, 1.0):
        left, keep = drop(ids, share, E)
        left[0, k - 1], keep[0, k - 1] = -1, False
        got = route_bwd(M, dw, l, left, score, renorm, 2.5)
        want = route_bwd(M, dw * keep, l, ids, score, renorm, 2.5)
        assert torch.equal(got, want)
        d, dm = O.router_bwd(O.np64(dw * keep), O.np64(l), ids.cpu().numpy(), score, renorm, 2.5)
        O.check(got, d, dm, 2 * exp_ops(O.np64(l), E) + k, "dlogits")
    assert M.mhc_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_choice_is_found_again_among_ties_and_close_logits(M, score):
    """Ties, logits that differ in their last bits, masked experts, and kept
    slots in another order."""
    g, k, E = rng(7), 6, 64
    close = torch.stack([torch.randperm(E, generator=g) for _ in range(8)]).int()
    l = torch.cat(((torch.tensor(1.0).view(torch.int32) + close).view(torch.float32),
                   torch.randint(0, 4, (8, E), generator=g).float(),
                   torch.where(torch.rand(8, E, generator=g) < 0.95, -torch.inf,
                               torch.randn(8, E, generator=g)))).cuda()
    ids, _ = route(M, l, k, score, True)
    dw = torch.randn(len(l), k, generator=g).cuda()
    left, keep = drop(ids, 0.4, 3)
    left[:, 2], keep[:, 2] = -1, False
    want = route_bwd(M, dw * keep, l, ids, score, True)
    assert torch.equal(route_bwd(M, dw, l, left, score, True), want)
    assert M.mhc_device_error() == 0
    turn = torch.argsort(torch.rand(len(l), k, generator=g), dim=1).cuda()
    got = route_bwd(M, dw.gather(1, turn), l, left.gather(1, turn).contiguous(), score, True)
    assert torch.equal(got, want) and M.mhc_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ids_that_are_not_the_choice_are_left_out_and_reported(M, score):
    """The weights' sum cannot be found again for a row with a dropped slot and
    an expert that the forward did not choose."""
    l = torch.tensor([[5.0, 4, 3, 2, 1, 0]] * 2, device="cuda")
    dw = torch.tensor([[1.0, -2, 4]] * 2, device="cuda")
    ids = lambda *v: torch.tensor([[0, 1, 2], v], dtype=torch.int32, device="cuda")  # noqa: E731
    got = route_bwd(M, dw, l, ids(0, 4, -1), score, True)
    assert M.mhc_device_error() == 204 and M.mhc_device_error() == 0
    want = route_bwd(M, torch.tensor([[1.0, -2, 4], [1, 0, 0]], device="cuda"), l, ids(0, 1, 2),
                     score, True)
    assert torch.equal(got, want) and M.mhc_device_error() == 0
    # every slot kept: any choice has its gradient, and so have plain weights
    got = route_bwd(M, dw, l, ids(0, 4, 5), score, True)
    d, dm = O.router_bwd(O.np64(dw), O.np64(l), np.array([[0, 1, 2], [0, 4, 5]]), score, True, 1.0)
    O.check(got, d, dm, 2 * exp_ops(O.np64(l), 6) + 3, "dlogits")
    route_bwd(M, dw, l, ids(0, 4, -1), score, False)
    assert M.mhc_device_error() == 0
