"""A tile whose sum runs for most of a second is waited for, not given up."""
import pytest
import torch

from tests import plain64 as p64
from tests import test_gpu_gate_up as base
from weight_only_quantized_qmm_b200 import api

pytestmark = pytest.mark.gpu


def test_parameter_gradients_of_very_many_tokens():
    # one token in 4096 counts: the sums are integers up to 2^15, exact in fp32 in any order.
    # (Not many small terms: the tensor cores cut each product at about 2^-26 of the
    # accumulator, so equal ones stop adding at 2^26 of them.)
    M, K, N = 1 << 27, 32, 8
    w = base.weight(N, K, 4, 32, torch.bfloat16, 1)
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dy[::4096] = 1.0
    _, ds, dz = api.qmm_matmul_backward(dy, x, w, need_dx=False, g_dtype=torch.float32)
    q, _ = p64.dequant64(w)
    assert (dz == 2.0 ** 15 * K).all()
    assert torch.equal(ds.double(), 2.0 ** 15 * p64.by_group(q, 32))
    del x, dy
    torch.cuda.empty_cache()
