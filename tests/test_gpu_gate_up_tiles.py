"""The products of packed weights where every CTA (pair) takes several tiles:
operand and code rings, scale windows and the two accumulators carried from tile
to tile, and the staged stores.  Against 64-bit forms, in guarded buffers."""
import pytest
import torch

from tests import plain64 as p64
from tests import test_gpu_gate_up as base
from tests.helpers import Guarded
from weight_only_quantized_qmm_b200 import _lib, api

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def tiles_each(M, cols, tile_cols, parts=1):
    """Tiles of the busiest CTA pair, for tiles of 256 rows.  (Single CTAs take
    tiles of 128 rows, and there are twice as many of them as pairs: as many
    tiles or more.)"""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    tiles = parts * -(-M // 256) * -(-cols // tile_cols)
    return -(-tiles // pairs)


def dense_first(call, M, K, N, bits):
    """Whether the call dequantizes its weights beforehand, from its workspace."""
    need = getattr(_lib.load(), call + "_workspace_bytes")(M, K, N, bits)
    own = {"qmm_gate_up_silu": 0, "qmm_matmul_backward": 2 * M * -(-N // 8) * 8 if N % 8 else 0,
           "qmm_gate_up_silu_backward": 4 * M * -(-N // 8) * 8}[call]
    return need > own + 16


# (M, K, F, bits, gs, dequantized first): dense with many and few steps a tile, F a multiple
# of 8 and odd, ragged tokens; codes in the kernel with several windows of 8 groups a tile
# (scales by TMA), with scales from global memory, 3-bit codes (two steps a box), and up to
# 128 tokens (single CTAs)
@pytest.mark.parametrize("M,K,F,bits,gs,dense", [
    (5000, 2048, 3000, 4, 64, True), (2601, 1056, 2893, 3, 32, True), (5000, 96, 1500, 3, 32, True),
    (600, 2048, 10000, 4, 64, False), (520, 1024, 13001, 6, 32, False), (300, 1280, 14336, 3, 64, False),
    (700, 2048, 9600, 8, 128, False), (530, 320, 13000, 2, 64, False), (130, 512, 29000, 4, 32, False),
    (100, 512, 57000, 4, 32, False), (60, 1024, 57001, 2, 128, False)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward(M, K, F, bits, gs, dense, dtype):
    assert dense_first("qmm_gate_up_silu", M, K, F, bits) == dense
    assert tiles_each(M, F, 128) >= 3
    base.check_forward(M, bits, gs, K, F, dtype)


# dx: (M, K, N, bits, gs, dequantized first); a cluster's third and fifth tile, one step a tile
# and many, two parts, scales by TMA and not
@pytest.mark.parametrize("M,K,N,bits,gs,dense", [
    (5200, 4096, 1400, 4, 64, True), (2611, 4064, 200, 3, 32, True), (5000, 4064, 50, 3, 32, True),
    (4700, 4096, 320, 4, 64, False), (2700, 4096, 60, 2, 32, False), (2600, 4096, 333, 6, 128, False),
    (2609, 4224, 130, 8, 64, False), (2600, 4096, 200, 3, 32, False)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_dx(M, K, N, bits, gs, dense, dtype):
    assert dense_first("qmm_matmul_backward", M, K, N, bits) == dense
    assert tiles_each(M, K, 256) >= 3
    w = base.weight(N, K, bits, gs, dtype, 4)
    dy = base.act(M, N, 6, dtype, 0.1)
    dx = Guarded((M, K), dtype)
    api.qmm_matmul_backward(dy, base.act(M, K, 5, dtype), w, need_params=False, dx=dx.out)
    want, bound = p64.dx64([dy.double()], [w], F32, dtype)
    p64.close(dx.check(), want, p64.rounded(bound, want, dtype), "dx")


# the parameter gradients: a pair's third to sixth tile, one step of ragged tokens and many
@pytest.mark.parametrize("M,K,N,bits,gs", [(2600, 4096, 3500, 4, 64), (700, 4096, 6001, 6, 32), (70, 4064, 5000, 3, 32),
                                           (9, 3584, 7777, 8, 128), (330, 4128, 3900, 2, 32)])
@pytest.mark.parametrize("dtype,g_dtype", [(BF, F32), (HF, HF)])
def test_parameters(M, K, N, bits, gs, dtype, g_dtype):
    assert tiles_each(N, K, 256) >= 3
    w = base.weight(N, K, bits, gs, dtype, 4)
    x, dy = base.act(M, K, 5, dtype), base.act(M, N, 6, dtype, 0.1)
    G = K // gs
    ds, dz = Guarded((N, G), g_dtype), Guarded((N, G), g_dtype)
    api.qmm_matmul_backward(dy, x, w, need_dx=False, dscales=ds.out, dbiases=dz.out)
    wants, bounds = p64.params64(dy.double(), x, w, F32)
    for got, wt, b, n in zip((ds, dz), wants, bounds, ("dscales", "dbiases")):
        p64.close(got.check(n), wt, p64.rounded(b, wt, g_dtype), n)


@pytest.mark.parametrize("M,K,F,bits,gs,dense", [(5200, 4096, 700, 4, 64, True), (2700, 4096, 130, 4, 32, False)])
@pytest.mark.parametrize("dtype,g_dtype", [(BF, F32), (HF, HF)])
def test_gated_backward(M, K, F, bits, gs, dense, dtype, g_dtype):
    assert dense_first("qmm_gate_up_silu_backward", M, K, F, bits) == dense
    assert tiles_each(M, K, 256) >= 3
    base.check_gated_backward(M, bits, gs, K, F, dtype, g_dtype)


def test_gated_backward_wide():
    """Both parts' parameter gradients over many tiles, and dx over a long sum."""
    M, K, F = 300, 4096, 3900
    assert tiles_each(F, K, 256, 2) >= 6
    base.check_gated_backward(M, 4, 64, K, F, BF, F32)
