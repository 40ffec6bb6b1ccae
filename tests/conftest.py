import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built extension")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle
    oracle.lib()
    return oracle


@pytest.fixture(scope="session", autouse=True)
def _warm_torch_math():
    """In about one process of fifty the first f64 logsumexp that torch spreads
    over its threads is good to 1e-10 only in one thread's part (its logits and
    every later call are right to the last bits): let that call be this one."""
    import torch
    torch.logsumexp(torch.rand(512, 512, dtype=torch.float64), dim=-1)
