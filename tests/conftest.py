import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# CPU tests of refusals whose sizes just inside a limit pass every check, with addresses that are no memory:
# without a GPU the call ends at the device check, with one it would launch.
LAUNCH_ON_A_GPU = {"test_attn_refuses_more_prefix_work_than_one_call_holds"}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built CUDA library")


def pytest_runtest_setup(item):
    if item.name in LAUNCH_ON_A_GPU:
        import torch

        if torch.cuda.is_available():
            pytest.skip("would launch on addresses that are no memory: runs without a GPU only")
