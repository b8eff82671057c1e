"""Calls repeat bit for bit, also while other work holds the memory system: the
kernels' copies then land late and out of order.  The first result is checked
against the 64-bit forms."""
import pytest
import torch

from tests import plain64 as p64
from tests import test_gpu_gate_up as base
from weight_only_quantized_qmm_b200 import api

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def repeats(call, times=150):
    """`call` gives the bits of its first result: by itself, after kernels that leave
    the caches full, and beside a stream of copies."""
    first = [t.clone() for t in call()]
    src = torch.zeros(96 << 20, dtype=torch.uint8, device="cuda")
    dst, other = torch.empty_like(src), torch.cuda.Stream()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(times):
        if i % 3 == 1:
            dst.copy_(src)
        if i % 3 == 2:
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                for _ in range(3):
                    dst.copy_(src)
        for a, b in zip(first, call()):
            wrong += (a.view(torch.int16 if a.element_size() == 2 else torch.int32)
                      != b.view(torch.int16 if b.element_size() == 2 else torch.int32)).any()
    torch.cuda.synchronize()
    assert int(wrong) == 0, f"{int(wrong)} outputs of {times} calls differ from the first call's"
    return first


# every width: codes dequantized in the kernel, on pairs and on single CTAs, sums split and
# whole, scales by TMA (K / gs a multiple of 8) and not
@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("M,K,F,gs", [(24, 1792, 1100, 128), (24, 2048, 9000, 64), (200, 2176, 1100, 128),
                                      (200, 2048, 8000, 32), (600, 1152, 5000, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward(bits, M, K, F, gs, dtype):
    gate, up = base.weight(F, K, bits, gs, dtype, 1), base.weight(F, K, bits, gs, dtype, 2)
    x = base.act(M, K, 3, dtype)
    h, g, u = repeats(lambda: api.qmm_gate_up_silu(x, gate, up, save=True))
    want, bound = p64.gate_up64(x, gate, up, dtype)
    for got, w, b in zip((h, g, u), want, bound):
        p64.close(got, w, p64.rounded(b, w, dtype), "forward")


@pytest.mark.parametrize("bits", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("M,K,N,gs", [(1, 3968, 3558, 128), (40, 2048, 3000, 32), (200, 4096, 4096, 64),
                                      (700, 3712, 2500, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_backward(bits, M, K, N, gs, dtype):
    w = base.weight(N, K, bits, gs, dtype, 4)
    x, dy = base.act(M, K, 5, dtype), base.act(M, N, 6, dtype, 0.1)
    dx, ds, dz = repeats(lambda: api.qmm_matmul_backward(dy, x, w, g_dtype=F32))
    alone, _, _ = repeats(lambda: (api.qmm_matmul_backward(dy, x, w, need_params=False)[0],) * 3, 50)
    assert torch.equal(alone, dx)
    want, bound = p64.dx64([dy.double()], [w], F32, dtype)
    p64.close(dx, want, p64.rounded(bound, want, dtype), "dx")
    wants, bounds = p64.params64(dy.double(), x, w, F32)
    for got, wt, b in zip((ds, dz), wants, bounds):
        p64.close(got, wt, p64.rounded(b, wt, F32), "parameters")


@pytest.mark.parametrize("bits", [3, 4, 6])
def test_gated_backward(bits):
    M, K, F, gs = 90, 1664, 2000, 128
    gate, up = base.weight(F, K, bits, gs, BF, 1), base.weight(F, K, bits, gs, BF, 2)
    x, dh, g, u = base.act(M, K, 3, BF), base.act(M, F, 4, BF, 0.1), base.act(M, F, 5, BF), base.act(M, F, 6, BF)

    def call():
        dx, dg, du = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up)
        return dx, *dg, *du

    dx = repeats(call)[0]
    want, bound = p64.dx64(p64.act_grad64(dh, g, u), [gate, up], BF, BF)
    p64.close(dx, want, p64.rounded(bound, want, BF), "dx")


@pytest.mark.parametrize("n,rows,cols", [(300, 5000, 1024), (1500, 400, 1024), (9000, 30000, 512)])
def test_table_gradient(n, rows, cols):
    qw = base.weight(rows, cols, 4, 64, BF, 1)
    ids = torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()
    dy = base.act(n, cols, 2, BF)
    repeats(lambda: api.qmm_embedding_backward(dy, ids, qw, 2.0, F32))
