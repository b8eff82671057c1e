"""Empty batches of the gradient calls: what is not asked for and what holds no
elements are both null addresses, and neither is an error."""
import ctypes

import pytest
import torch

from weight_only_quantized_qmm_b200 import _lib, api
from weight_only_quantized_qmm_b200 import workloads as wl

A = 0x10000  # an aligned fake device address: never dereferenced by these calls
BF = _lib.QMM_BF16


def calls(L):
    def one(M, rows, dx, grads):
        w = _lib.QWeightC(A, A, A, BF, rows, 128, 64, 4, 0)
        return L.qmm_matmul_backward(A, A, BF, M, 128, ctypes.byref(w), dx, *grads[:2], BF, A, 1 << 40, None)

    def two(M, rows, dx, grads):
        w = _lib.QWeightC(A, A, A, BF, rows, 128, 64, 4, 0)
        return L.qmm_gate_up_silu_backward(A, A, A, A, BF, M, 128, ctypes.byref(w), ctypes.byref(w), dx, *grads, BF, A,
                                           1 << 40, None)

    return one, two


def test_nothing_to_write():
    none, some = (None,) * 4, (A,) * 4
    for call in calls(_lib.load()):
        assert call(0, 8, None, none) == _lib.QMM_OK  # dx of no tokens
        assert call(0, 8, A, none) == _lib.QMM_OK
        assert call(2, 0, None, none) == _lib.QMM_OK  # the parameters of no rows
        assert call(2, 0, None, some) == _lib.QMM_OK
        assert call(2, 8, None, none) == _lib.QMM_ERR_INVALID_ARG
        assert call(0, 8, None, (A, None, A, A)) == _lib.QMM_ERR_INVALID_ARG
        assert call(-1, 8, None, none) == _lib.QMM_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 41])
def test_binding_without_tokens(rows):
    gate, up = (api.qmm_quantize(wl.gen_weight(rows, 128, s).cuda(), 64, 4, torch.bfloat16) for s in (1, 2))
    x, h = (torch.zeros(0, n, dtype=torch.bfloat16, device="cuda") for n in (128, rows))
    for shape in ((0,), (3, 0)):
        xs, hs = x.view(*shape, 128), h.view(*shape, rows)
        dx, ds, dz = api.qmm_matmul_backward(hs, xs, gate, need_params=False)
        assert dx.shape == xs.shape and ds is None and dz is None
        dx, dg, du = api.qmm_gate_up_silu_backward(hs, xs, hs, hs, gate, up, need_params=False)
        assert dx.shape == xs.shape and dg is None and du is None
        dx, ds, dz = api.qmm_matmul_backward(hs, xs, gate, need_dx=False)
        assert dx is None and (ds == 0).all() and (dz == 0).all()
        dx, dg, du = api.qmm_gate_up_silu_backward(hs, xs, hs, hs, gate, up, need_dx=False)
        assert dx is None and all((t == 0).all() for t in (*dg, *du))
