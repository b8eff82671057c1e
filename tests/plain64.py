"""Packed-weight operators in 64 bits on the GPU, written from their formulas,
with the elementwise error bounds that the kernels' roundings allow.

U[t] is half a rounding step of type t relative to the value.  The kernels
round each dequantized weight once to the activations' type (more than 16
tokens), dg and du of the gated block once, and each output once.  Sums run in
fp32: over n terms the tensor cores carry a chain of n / 16 additions, each off
by at most 2^-23 of the magnitudes' sum (they may truncate), which is E32 =
2^-14 with room for the 16 products of a step at the n <= 4096 used here."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least subnormal
E32 = 2.0 ** -14


def codes64(packed, cols, bits):
    """[rows, cols] codes: digit k of code i is bit i * bits + k of the row."""
    digits = torch.stack([(packed >> k) & 1 for k in range(32)], -1).reshape(packed.shape[0], cols, bits)
    return sum(digits[..., k].double() * 2.0 ** k for k in range(bits))


def dequant64(qw):
    """(q, w): codes and values of an affine QWeight."""
    q = codes64(qw.packed.view(qw.rows, -1), qw.cols, qw.bits)
    rep = lambda t: t.double().view(qw.rows, -1).repeat_interleave(qw.group_size, 1)  # noqa: E731
    return q, q * rep(qw.scales) + rep(qw.biases)


def by_group(t, gs):
    return t.unflatten(1, (-1, gs)).sum(2)


def rounded(bound, value, dtype):
    """`bound` on a sum's error, then one rounding of the result to dtype."""
    return bound + U[dtype] * (value.abs() + bound) + TINY[dtype]


def gate_up64(x, gate, up, w_type):
    """(h, g, u) and the bounds of their errors before the output's rounding;
    w_type: the type each weight is rounded to (float32: not rounded)."""
    X = x.double()
    out, err = [], []
    for w in (gate, up):
        _, W = dequant64(w)
        mag = X.abs() @ W.abs().t()
        out.append(X @ W.t())
        err.append(mag * (U[w_type] + E32) + TINY[w_type] * X.abs().sum(1, keepdim=True))
    g, u = out
    dg, du = err
    silu = g * torch.sigmoid(g)
    # |SiLU'| < 1.1; fp32 exp, division and products: a few parts in 2^22
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * 2.0 ** -20
    return (h, g, u), (dh, dg, du)


def act_grad64(dh, g, u):
    dh, g, u = dh.double(), g.double(), u.double()
    p = torch.sigmoid(g)
    return dh * u * p * (1 + g * (1 - p)), dh * g * p


def dx64(dys, ws, y_type, w_type):
    """Sum of dy . W over the pairs and its error bound: each dy rounded to
    y_type (float32: exact as given), each weight to w_type."""
    total = bound = 0.0
    for dy, w in zip(dys, ws):
        _, W = dequant64(w)
        u = U[y_type] + U[w_type] + E32 if y_type != torch.float32 else U[w_type] + E32
        total = total + dy @ W
        bound = (bound + dy.abs() @ W.abs() * (u + U[y_type] * U[w_type] + 2.0 ** -20)
                 + TINY[w_type] * dy.abs().sum(1, keepdim=True) + TINY[y_type] * W.abs().sum(0))
    return total, bound


def params64(dy, x, w, y_type):
    """(dscales, dbiases) and their bounds; dy rounded to y_type (float32: exact as given)."""
    q, _ = dequant64(w)
    X = x.double()
    dW, mag = dy.t() @ X, dy.abs().t() @ X.abs()
    u = (0.0 if y_type == torch.float32 else U[y_type] + 2.0 ** -20) + E32
    bound = mag * u + (0.0 if y_type == torch.float32 else TINY[y_type] * X.abs().sum(0))
    gs = w.group_size
    return ((by_group(dW * q, gs), by_group(dW, gs)),
            (by_group(bound * q + (mag * q) * E32, gs), by_group(bound + mag * E32, gs)))


def close(got, want, bound, what=""):
    """Every element within its bound, and where the result has a norm, the
    whole within 5e-3 of it."""
    got = got.double().reshape(want.shape)
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values are not finite"
    err = (got - want).abs()
    over = err > bound
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} past the bound, worst "
                            f"{float((err / bound.clamp_min(1e-300)).max()):.2f} times it")
    norm = float(want.norm())
    if norm > 0:
        assert float(err.norm()) <= 5e-3 * norm, f"{what}: {float(err.norm()) / norm:.2e} of the norm"
