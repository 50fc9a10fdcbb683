"""The example notices what its calls report: labels out of range (a vocabulary
that does not fit, padding other than ``ignore_index``) end its training."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("label", [64, -100])
def test_a_label_out_of_range(label):
    from ctc_prefix_beam_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("frame_head", os.path.join(ROOT, "examples", "frame_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    plain, calls = m.utterances, []

    def utterances(*args):
        x, targets, lens, seqs = plain(*args)
        calls.append(0)
        if len(calls) == 3:  # of the second step
            targets[1, 5] = label
        return x, targets, lens, seqs

    m.utterances = utterances
    with pytest.raises(RuntimeError, match="out of range"):
        m.main(steps=3, verbose=False)
    assert len(calls) == 3
