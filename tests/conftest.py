import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running case")


# Walks whose expected values are wrong, and why.  Strict: one that passes again is reported.
WRONG_VALUES = {
    "test_pages_follow_the_model[30-600-32-9000-3]":
        "the model appends to a page that another sequence holds: in step 13 token 6351 of sequence 3 goes to slot 15 "
        "of page 525, which holds token 6351 of sequence 0",
    "test_pages_follow_the_model[1500-4-16-5000-4]":
        "the model appends to a page that another sequence holds: in step 24 sequence 1074 is not among the refused, "
        "though its token 17 would go to slot 1 of page 1139, which holds token 17 of sequence 1204",
}


def pytest_collection_modifyitems(config, items):
    for item in items:
        if item.name in WRONG_VALUES:
            item.add_marker(pytest.mark.xfail(reason=WRONG_VALUES[item.name], strict=True, raises=AssertionError))
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
