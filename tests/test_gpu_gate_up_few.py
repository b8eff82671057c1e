"""The gated projection of up to 16 tokens at every width and group size, on rows
that the streaming kernel does not take: fewer than 16 rows, short rows, rows whose
groups are no multiple of 8."""
import pytest
import torch

from tests import test_gpu_gate_up as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("M,dtype", [(1, torch.float16), (3, torch.bfloat16), (8, torch.float16), (9, torch.bfloat16),
                                     (13, torch.float16), (16, torch.bfloat16)])
def test_forward(M, dtype, bits, gs):
    for K, F in ((gs, 1), (gs * 3, 7), (gs * 9, 100), (3328, 6), (1664, 1001), (16384, 40)):
        base.check_forward(M, bits, gs, K, F, dtype)
