"""Host tests that hand fake addresses past the library's checks are not run
where a GPU would take them."""
import types

import pytest
import torch

from tests import conftest, test_abi_host


@pytest.mark.parametrize("there", [True, False])
def test_fake_addresses_stay_off_a_gpu(monkeypatch, there):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: there)
    skipped = 0
    for name in vars(test_abi_host):
        try:
            conftest.pytest_runtest_setup(types.SimpleNamespace(originalname=name))
        except pytest.skip.Exception:
            skipped += 1
    assert hasattr(test_abi_host, "test_validation_errors_without_gpu")
    assert skipped == (2 if there else 0)
