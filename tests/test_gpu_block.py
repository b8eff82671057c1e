"""One fine-tuning step of a packed model's feed-forward path as it is used:
lookup, gated projection, down projection, and back to the table's scales and
biases, against the same step in 64 bits."""
import pytest
import torch

from tests import plain64 as p64
from weight_only_quantized_qmm_b200 import api
from weight_only_quantized_qmm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [1, 12, 70, 333])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step(T, dtype):
    V, D, F, gs = 400, 256, 608, 32
    quant = lambda n, k, bits, seed: api.qmm_quantize(wl.gen_weight(n, k, seed, 0.1).to(DEV), gs, bits, dtype)  # noqa: E731
    table, gate, up, down = quant(V, D, 6, 1), quant(F, D, 4, 2), quant(F, D, 4, 3), quant(D, F, 4, 4)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, 40, (T,), generator=g, dtype=torch.int32).to(DEV)
    alpha = 16.0
    dy = wl.gen_x(T, D, 5, "f32").to(dtype).to(DEV)

    x = api.qmm_embedding(ids, table, alpha)
    h, gp, up_ = api.qmm_gate_up_silu(x, gate, up, save=True)
    y = api.qmm_matmul(h, down)
    dh, dds, ddz = api.qmm_matmul_backward(dy, h, down)
    dx, dgate, dup = api.qmm_gate_up_silu_backward(dh, x, gp, up_, gate, up)
    # (in f32: with alpha and codes up to 63 these sums pass 65504, the largest f16)
    dts, dtz = api.qmm_embedding_backward(dx, ids, table, alpha, g_dtype=torch.float32)

    leaves = {}
    def w64(name, qw):
        q, _ = p64.dequant64(qw)
        s, z = (t.double().clone().requires_grad_() for t in (qw.scales, qw.biases))
        leaves[name] = (s, z)
        return q * s.repeat_interleave(gs, 1) + z.repeat_interleave(gs, 1)

    X = w64("table", table)[ids.long()] * alpha
    G, U = X @ w64("gate", gate).t(), X @ w64("up", up).t()
    Y = (G * torch.sigmoid(G) * U) @ w64("down", down).t()
    Y.backward(dy.double())
    # roundings in 16 bits along the way, each at most U relative to its value: x, three
    # weights, g, u, h, dh, dg and du, dx, the output: 12 at most on one path; errors of
    # independent terms add in squares, a cancelling sum by at most the same again
    tol = 12 * p64.U[dtype]
    pairs = [(y, Y), (dds, leaves["down"][0].grad), (ddz, leaves["down"][1].grad),
             (dgate[0], leaves["gate"][0].grad), (dgate[1], leaves["gate"][1].grad),
             (dup[0], leaves["up"][0].grad), (dup[1], leaves["up"][1].grad),
             (dts, leaves["table"][0].grad), (dtz, leaves["table"][1].grad)]
    for i, (got, want) in enumerate(pairs):
        want = want.detach()
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= tol, (i, rel)
