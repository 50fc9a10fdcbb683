"""An ignore_index that is no int32 value is refused, not cut to 32 bits."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("index", [1 << 32, -(1 << 32), (1 << 32) - 1, 1 << 31, -(1 << 31) - 1, 1 << 64])
def test_out_of_int32(index):
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    x, w = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(5, 16, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    one, lse = torch.ones((), device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        head.cross_entropy(x, w, t, ignore_index=index)
    with pytest.raises(ValueError):
        head.cross_entropy_backward(one, x, w, t, lse, ignore_index=index)
    for index in (-(1 << 31), (1 << 31) - 1, -100):
        head.cross_entropy(x, w, t, ignore_index=index)
