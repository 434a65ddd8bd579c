import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


@pytest.fixture(scope="session")
def oracle():
    import oracle as _oracle
    _oracle.build()
    return _oracle


@pytest.fixture(scope="session", autouse=True)
def _torch_exp_set_up():
    """torch's fp64 exp on the CPU sets itself up at its first use.  Where that use is
    spread over several threads, some processes get one thread's share off by 1e-10, which
    the oracle's comparisons at 1e-12 see; so the first use has one thread."""
    import torch
    torch.exp(torch.linspace(-1, 1, 64, dtype=torch.float64))
