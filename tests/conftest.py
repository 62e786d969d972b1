import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs the CUDA library)")
    config.addinivalue_line("markers", "slow: full-size workload (minutes on the oracle)")


def pytest_runtest_setup(item):
    # The tests of this name hand fake addresses past every check, down to the
    # one for a device: with a GPU there, the call would be made.
    if item.originalname.endswith("_without_gpu"):
        import torch
        if torch.cuda.is_available():
            pytest.skip("for machines without a GPU: its addresses are not real")


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.build()
    return oracle
