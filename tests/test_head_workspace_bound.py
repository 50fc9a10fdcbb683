"""The memory that the header promises for the gradients of the cross entropy
(no GPU needed: size queries only)."""
import pytest
import torch

from ctc_prefix_beam_gb300 import build as B
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    D.lib()


@pytest.mark.parametrize("n,v", [(1, 1), (8192, 65536), (16000, 5000), (524288, 4096), (524289, 193), (1 << 20, 32768),
                                 (1 << 24, 256), (1 << 24, 1 << 20)])
def test_pieces_of_the_vocabulary(n, v):
    """d: 256 MB, or 512 bytes a row; beside it, for rows rounded up to 256: x, the
    running dx (float32) and w; 16 bytes a row and the column sums of a piece (a
    16th of d's bytes); and the shares of a wave (152 SMs, 2 of 128 x 64 floats, twice)."""
    h = 64
    rows = -(-n // 256) * 256
    d = max(256 << 20, 512 * rows)
    most = d + d // 16 + rows * (2 * h + 4 * h + 32) + 2 * v * h + 2 * 2 * 152 * 128 * 64 * 4 + (1 << 16)
    assert head.cross_entropy_workspace_size(BF, n, v, h, True) <= most
