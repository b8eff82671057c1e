"""SiLU and its slope over the whole range of the pre-activation, against 64
bits: inputs for which every product and sum is exact, so that what is measured
is the activation alone."""
import pytest
import torch

from tests import plain64 as p64
from tests.helpers import Guarded
from weight_only_quantized_qmm_b200 import api

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def constant_rows(values, K, bits, gs, dtype):
    """A weight whose row n holds values[n] in every column."""
    n = values.numel()
    z = values.to(dtype).view(n, 1).expand(n, K // gs).contiguous().cuda()
    assert torch.equal(z[:, 0].cpu().double(), values.double())
    packed = torch.zeros(n, K * bits // 32, dtype=torch.int32, device="cuda")
    return api.QWeight(packed, torch.zeros_like(z), z, n, K, gs, bits)


# 4-bit rows in the kernel, 3-bit rows off 16 bytes dequantized first; sums split over a
# cluster, one tile a CTA (pair), and several; stores of whole rows and of staged ones
@pytest.mark.parametrize("M,K,F,bits,gs", [(20, 128, 96, 4, 64), (40, 1024, 90, 4, 64), (120, 128, 40001, 4, 128),
                                           (700, 128, 9000, 4, 32), (50, 96, 201, 3, 32), (600, 96, 17001, 3, 32)])
@pytest.mark.parametrize("dtype,out", [(BF, F32), (HF, F32), (BF, BF)])
def test_forward(M, K, F, bits, gs, dtype, out):
    # x = 1 + m/128 and w = -n/128 of 8 bits each: every partial sum is a multiple of 2^-14
    # below 2^24 of them for K = 128; g runs from 0 to about -206 (K = 1024: n/1024 instead)
    a = 1.0 + (torch.arange(M) % 128).double() / 128
    n = (torch.arange(F) % 104).double()
    x = a.view(M, 1).expand(M, K).to(dtype).contiguous().cuda()
    gate = constant_rows(-n / max(K, 128), K, bits, gs, dtype)
    up = constant_rows(torch.full((F,), 1.0 / max(K, 128), dtype=torch.float64), K, bits, gs, dtype)
    share = K / max(K, 128)
    g = (-a.view(M, 1) * n * share).cuda()
    u = (a.view(M, 1) * share).cuda().expand(M, F)
    h = g * torch.sigmoid(g) * u
    # f32: e^-|g| within one step (2^-23 of it, or 2^-149), 1 + it half of one, the quotient two,
    # the three products half of one each: 5 * 2^-23 < 2^-20.  16 bits: the fast exponential, whose
    # error is 2 + 1.173 |g| steps, 124 where e^-|g| is not zero (|g| < 104): 129 * 2^-23 < 2^-15
    rel = 2.0 ** (-20 if out is F32 else -15)
    bound = h.abs() * rel + (1 + g.abs()) * (1 + u) * 2.0 ** -148
    o, pre = Guarded((M, F), out), (Guarded((M, F), dtype), Guarded((M, F), dtype))
    api.qmm_gate_up_silu(x, gate, up, out=o.out, g_pre=pre[0].out, u_pre=pre[1].out)
    p64.close(pre[0].check(), g, p64.rounded(0 * g, g, dtype), "g")
    p64.close(pre[1].check(), u, p64.rounded(0 * u, u, dtype), "u")
    p64.close(o.check(), h, p64.rounded(bound, h, out), "h")


@pytest.mark.parametrize("F", [2048, 1999])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient(F, dtype):
    """One token and x = 1: the bias gradients of a group of 32 are 32 dg and 32 du."""
    K, gs = 64, 32
    w = constant_rows(torch.ones(F, dtype=torch.float64), K, 4, gs, dtype)
    x = torch.ones(1, K, dtype=dtype, device="cuda")
    g = (torch.arange(F).double() * (200.0 / F) - 110.0).to(dtype).view(1, F).cuda()
    dh = torch.full((1, F), 1.5, dtype=dtype, device="cuda")
    u = torch.full((1, F), -0.75, dtype=dtype, device="cuda")
    out = [Guarded((F, K // gs), F32) for _ in range(4)]
    api.qmm_gate_up_silu_backward(dh, x, g, u, w, w, need_dx=False, dgate=(out[0].out, out[1].out),
                                  dup=(out[2].out, out[3].out), g_dtype=F32)
    G, D, Up = g.double(), dh.double(), u.double()
    p, q = torch.sigmoid(G), torch.sigmoid(-G)
    for got, want, mag in ((out[1], D * Up * p * (1 + G * q), (D * Up).abs() * p * (1 + G.abs() * q)),
                           (out[3], D * G * p, (D * G).abs() * p)):
        # p and 1 - p within 128 * 2^-23 of themselves (the fast exponential: 124), then at most
        # eight half steps; the slope's two terms may cancel, so relative to their magnitudes;
        # one rounding to 16 bits
        bound = p64.rounded(mag * 2.0 ** -15 + (1 + G.abs()) * 2.0 ** -147, want, dtype)
        want, bound = (32 * t.view(F, 1).expand(F, K // gs) for t in (want, bound))
        p64.close(got.check(), want, bound, "bias gradient")
