"""examples/decoder_block.py: every way that the gradient takes to the input is
there, once, however small its share of the whole."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATHS = [f"{layer}.{way}" for layer, ways in
         (("attn", ("q", "k", "v")), ("moe", ("router", "experts")))
         for way in ("H_pre", "H_post", "H_res", "aggregate", "residual") + ways]


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    return block


@pytest.mark.parametrize("kw", [{}, {"T": 65, "n": 8, "C": 264, "Hq": 6, "Hk": 3, "D": 40, "E": 5,
                                     "k": 3, "F": 72, "align": 8, "seed": 1}])
def test_every_path_of_the_gradient_counts_once(kw):
    """With R the part of dx that comes along one path (the reference's dx less the
    one with that path cut), dx = (the rest) + c R for some c, and c is 1; it is
    0 for a missing path and 2 for one taken twice.  The other errors of dx, less
    than a tenth of its norm, point anywhere in some 10^5 dimensions, of which
    10^3 would do: they move c by less than 0.1 / sqrt(10^3) over R's share of the
    norm, which is 1/6 for a share of 2%."""
    block = load()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s, p, x, dout = block.make(**kw)
    _, caches = block.forward(s, p, x)
    dx = block.backward(s, p, caches, dout)[0].float()
    assert block.M.mhc_device_error() == 0
    ids = caches[1][1]["ids"]
    wide = {**p, **{a: {n: t.float() for n, t in p[a].items()} for a in ("attn", "moe")}}

    def grad(cut=None):
        leaf = x.float().requires_grad_()
        out = block.reference(s, wide, leaf, ids, lambda path, v: v.detach() if path == cut else v)
        return torch.autograd.grad(out, leaf, dout.float())[0]

    whole = grad()
    for path in PATHS:
        R = whole - grad(path)
        share = float(R.norm() / whole.norm())
        assert share > 0.02, (path, share)
        c = 1 + float(((dx - whole) * R).sum() / R.square().sum())
        assert abs(c - 1) <= 1 / 6, (path, c, share)
