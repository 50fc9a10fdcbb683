"""The operators together as a user runs them: examples/frame_head.py trains a
head through them and decodes with it, offline and streaming."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_frame_head_example():
    from ctc_prefix_beam_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("frame_head", os.path.join(ROOT, "examples", "frame_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(steps=60, verbose=False)
    assert r["losses"][-1] < 0.25 * r["losses"][0]
    assert r["error_before"] > 0.5 and r["error_after"] < 0.1
    assert abs(r["error_streaming"] - r["error_after"]) < 0.02
