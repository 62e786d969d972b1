"""examples/decoder_block.py: the operators together, against autograd."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [{}, {"T": 65, "n": 8, "C": 264, "Hq": 6, "Hk": 3, "D": 40, "E": 5,
                                     "k": 3, "F": 72, "align": 8, "seed": 1}])
def test_block_gradients(kw):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    # a value on its way through both layers and back is rounded to bf16 about
    # two dozen times, each by at most 2^-8 of itself; a relu whose input is
    # that near zero may also switch, so twice that
    errs = block.compare(*block.make(**kw))
    bad = {n: e for n, e in errs.items() if not e <= 48 * 2.0 ** -8}
    assert not bad, bad
    assert block.M.mhc_device_error() == 0
