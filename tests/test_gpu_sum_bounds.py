"""Products whose fp32 sums are short or long, with a bound that follows the
summed length: n terms are n / 16 additions of 16 products into an accumulator,
each off by at most 2^-23 of the magnitudes' sum, and as much again as 16 of
them for the products of a step and the few additions after it (joined parts of
a sum, a group's columns)."""
import pytest
import torch

from tests import plain64 as p64
from tests import test_gpu_gate_up as base

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def bound_sums_of(monkeypatch, n):
    monkeypatch.setattr(p64, "E32", (n / 16 + 16) * 2.0 ** -23)


@pytest.mark.parametrize("bits,gs,K,rows", [(2, 32, 32, 40), (4, 64, 64, 33), (8, 32, 96, 70), (3, 32, 96, 130),
                                            (6, 128, 128, 90)])
@pytest.mark.parametrize("M", [17, 60, 129])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_short_sums(monkeypatch, M, bits, gs, K, rows, dtype):
    bound_sums_of(monkeypatch, K)
    base.check_forward(M, bits, gs, K, rows, dtype)
    bound_sums_of(monkeypatch, max(M, 2 * rows))
    base.check_matmul_backward(M, bits, gs, K, rows, dtype, F32)
    base.check_gated_backward(M, bits, gs, K, rows, dtype, F32)


def test_long_sums_of_inputs(monkeypatch):
    bound_sums_of(monkeypatch, 16384)
    for M in (33, 300):
        base.check_forward(M, 2, 128, 16384, 70, BF)
        base.check_forward(M, 4, 64, 16384, 300, HF)


@pytest.mark.parametrize("M", [20, 200])
def test_long_sums_of_rows(monkeypatch, M):
    bound_sums_of(monkeypatch, 20000)
    base.check_matmul_backward(M, 4, 32, 64, 20000, HF, F32)
    bound_sums_of(monkeypatch, 40000)
    base.check_gated_backward(M, 4, 32, 64, 20000, BF, F32)


def test_long_sums_of_tokens(monkeypatch):
    bound_sums_of(monkeypatch, 30001)
    base.check_matmul_backward(30001, 4, 64, 320, 100, BF, F32)
    base.check_gated_backward(30001, 6, 32, 160, 72, HF, F32)
