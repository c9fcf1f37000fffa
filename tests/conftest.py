import gc
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU and the built CUDA library")


def pytest_runtest_setup(item):
    # The device tensors of earlier tests that sit in reference cycles (the traceback of an expected error holds
    # its frame) are freed here, not by a collection in the middle of a test that compares allocated bytes.
    if item.get_closest_marker("gpu"):
        gc.collect()
