"""The dense gated projection and the backward passes of the quantized
products, against 64-bit forms."""
import pytest
import torch

from tests import plain64 as p64
from tests.helpers import Guarded
from weight_only_quantized_qmm_b200 import api
from weight_only_quantized_qmm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAME = {BF: "bf16", HF: "f16"}


def weight(rows, cols, bits, gs, dtype, seed):
    return api.qmm_quantize(wl.gen_weight(rows, cols, seed, 0.05).to(DEV), gs, bits, dtype)


def act(m, n, seed, dtype, std=1.0):
    return (wl.gen_x(m, n, seed, "f32") * std).to(dtype).to(DEV)


# (bits, gs, K, rows): every width and group size; rows and groups that fill no tile
SHAPES = [(2, 32, 32, 1), (2, 64, 448, 257), (3, 32, 96, 130), (3, 128, 384, 64), (4, 32, 2080, 77), (4, 64, 512, 384),
          (4, 128, 128, 1001), (6, 32, 160, 129), (6, 64, 1024, 100), (8, 32, 288, 65), (8, 128, 640, 200),
          (4, 64, 4096, 513)]


def check_forward(M, bits, gs, K, F, dtype):
    gate, up = weight(F, K, bits, gs, dtype, 1), weight(F, K, bits, gs, dtype, 2)
    x = act(M, K, 3, dtype)
    (h, g, u), (eh, eg, eu) = p64.gate_up64(x, gate, up, dtype)
    out16, out32 = Guarded((M, F), dtype), Guarded((M, F), F32)
    pre = Guarded((M, F), dtype), Guarded((M, F), dtype)
    api.qmm_gate_up_silu(x, gate, up, out=out32.out)
    api.qmm_gate_up_silu(x, gate, up, out=out16.out, g_pre=pre[0].out, u_pre=pre[1].out)
    p64.close(out32.check(), h, p64.rounded(eh, h, F32), "h f32")
    p64.close(out16.check(), h, p64.rounded(eh, h, dtype), "h")
    p64.close(pre[0].check(), g, p64.rounded(eg, g, dtype), "g")
    p64.close(pre[1].check(), u, p64.rounded(eu, u, dtype), "u")


@pytest.mark.parametrize("bits,gs,K,F", SHAPES)
@pytest.mark.parametrize("M,dtype", [(1, BF), (5, HF), (16, BF), (17, HF), (100, BF), (128, HF), (129, BF), (300, BF)])
def test_forward(M, dtype, bits, gs, K, F):
    check_forward(M, bits, gs, K, F, dtype)


def check_matmul_backward(M, bits, gs, K, N, dtype, g_dtype):
    w = weight(N, K, bits, gs, dtype, 4)
    x, dy = act(M, K, 5, dtype), act(M, N, 6, dtype, 0.1)
    G = K // gs
    dx, ds, dz = Guarded((M, K), dtype), Guarded((N, G), g_dtype), Guarded((N, G), g_dtype)
    api.qmm_matmul_backward(dy, x, w, dx=dx.out, dscales=ds.out, dbiases=dz.out)
    want, bound = p64.dx64([dy.double()], [w], F32, dtype)
    p64.close(dx.check(), want, p64.rounded(bound, want, dtype), "dx")
    wants, bounds = p64.params64(dy.double(), x, w, F32)
    for got, wt, b, n in zip((ds, dz), wants, bounds, ("dscales", "dbiases")):
        p64.close(got.check(n), wt, p64.rounded(b, wt, g_dtype), n)


@pytest.mark.parametrize("bits,gs,K,N", SHAPES)
@pytest.mark.parametrize("M,dtype,g_dtype", [(1, BF, F32), (7, HF, HF), (64, BF, BF), (129, HF, F32), (260, BF, F32)])
def test_matmul_backward(M, dtype, g_dtype, bits, gs, K, N):
    check_matmul_backward(M, bits, gs, K, N, dtype, g_dtype)


def check_gated_backward(M, bits, gs, K, F, dtype, g_dtype):
    gate, up = weight(F, K, bits, gs, dtype, 7), weight(F, K, bits, gs, dtype, 8)
    x, dh = act(M, K, 9, dtype), act(M, F, 10, dtype, 0.1)
    g, u = act(M, F, 11, dtype, 2.0), act(M, F, 12, dtype)
    G = K // gs
    dx = Guarded((M, K), dtype)
    out = [Guarded((F, G), g_dtype) for _ in range(4)]
    api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, dx=dx.out, dgate=(out[0].out, out[1].out),
                                  dup=(out[2].out, out[3].out))
    dg, du = p64.act_grad64(dh, g, u)
    want, bound = p64.dx64([dg, du], [gate, up], dtype, dtype)
    p64.close(dx.check(), want, p64.rounded(bound, want, dtype), "dx")
    for i, (d, w) in enumerate(((dg, gate), (du, up))):
        wants, bounds = p64.params64(d, x, w, dtype)
        for j in range(2):
            p64.close(out[2 * i + j].check(), wants[j], p64.rounded(bounds[j], wants[j], g_dtype), f"grad {i} {j}")


@pytest.mark.parametrize("bits,gs,K,F", SHAPES)
@pytest.mark.parametrize("M,dtype,g_dtype", [(1, HF, F32), (33, BF, BF), (128, HF, HF), (130, BF, F32)])
def test_gated_backward(M, dtype, g_dtype, bits, gs, K, F):
    check_gated_backward(M, bits, gs, K, F, dtype, g_dtype)


@pytest.mark.parametrize("M", [700, 1500])
def test_many_tokens(M):
    check_forward(M, 4, 64, 1088, 1400, BF)
    check_gated_backward(M, 4, 64, 1088, 1400, BF, F32)
    check_matmul_backward(M, 6, 32, 2080, 900, HF, F32)


def test_parts_of_the_gradient():
    """dx alone, the parameters alone, and both give the same bits; so does a
    second call, and a workspace that held something else."""
    M, K, F = 90, 320, 200
    gate, up = weight(F, K, 4, 64, BF, 1), weight(F, K, 4, 64, BF, 2)
    x, dh, g, u = act(M, K, 3, BF), act(M, F, 4, BF), act(M, F, 5, BF), act(M, F, 6, BF)
    both = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up)
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    again = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, workspace=ws)
    dx = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, need_params=False)
    pg = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, need_dx=False)
    assert dx[1] is None and dx[2] is None and pg[0] is None
    flat = lambda r: [r[0], *r[1], *r[2]]  # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(flat(both), flat(again)))
    assert torch.equal(both[0], dx[0]) and all(torch.equal(a, b) for a, b in zip(flat(both)[1:], [*pg[1], *pg[2]]))
    m = api.qmm_matmul_backward(dh, x, gate)
    assert torch.equal(m[0], api.qmm_matmul_backward(dh, x, gate, need_params=False)[0])
    n = api.qmm_matmul_backward(dh, x, gate, need_dx=False, workspace=ws)
    assert n[0] is None and torch.equal(m[1], n[1]) and torch.equal(m[2], n[2])


def test_no_tokens_and_shapes():
    gate, up = weight(40, 128, 4, 64, BF, 1), weight(40, 128, 4, 64, BF, 2)
    x0 = act(0, 128, 1, BF)
    h, g, u = api.qmm_gate_up_silu(x0, gate, up, save=True)
    assert h.shape == g.shape == u.shape == (0, 40)
    dx, dg, du = api.qmm_gate_up_silu_backward(h, x0, g, u, gate, up)
    assert dx.shape == (0, 128) and all((t == 0).all() for t in (*dg, *du))
    dx, ds, dz = api.qmm_matmul_backward(h, x0, gate)
    assert dx.shape == (0, 128) and (ds == 0).all() and (dz == 0).all()
    # leading dimensions are kept; a transposed view is taken as it reads
    x = act(6, 128, 1, BF)
    flat = api.qmm_gate_up_silu(x, gate, up)
    assert torch.equal(api.qmm_gate_up_silu(x.view(2, 3, 128), gate, up).view(6, 40), flat)
    assert torch.equal(api.qmm_gate_up_silu(x.t().contiguous().t(), gate, up), flat)


def test_not_finite_rows_stay_by_themselves():
    """A token with infinities or NaN spoils its own rows of h and dx only, and
    large pre-activations saturate as SiLU does."""
    M, K, F = 40, 256, 300
    gate, up = weight(F, K, 4, 64, BF, 1), weight(F, K, 4, 64, BF, 2)
    x = act(M, K, 3, BF)
    for m in (M, 9):
        y = x[:m].clone()
        y[3, 5], y[7, 0] = float("nan"), float("inf")
        keep = [i for i in range(m) if i not in (3, 7)]
        a, b = api.qmm_gate_up_silu(x[:m], gate, up), api.qmm_gate_up_silu(y, gate, up)
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[3]).all()
    dh, g, u = act(M, F, 4, BF), act(M, F, 5, BF), act(M, F, 6, BF)
    bad = dh.clone()
    bad[3, 7] = float("nan")
    a = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up)
    b = api.qmm_gate_up_silu_backward(bad, x, g, u, gate, up)
    keep = [i for i in range(M) if i != 3]
    assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][3]).all()
    rows = [i for i in range(F) if i != 7]
    for p, q in zip((*a[1], *a[2]), (*b[1], *b[2])):
        assert torch.equal(p[rows], q[rows]) and torch.isnan(q[7]).all()
    # SiLU and its slope at +-large g: g and 1, 0 and 0
    g[:, ::2], g[:, 1::2] = 200.0, -200.0
    dg, du = p64.act_grad64(dh, g, u)
    want, bound = p64.dx64([dg, du], [gate, up], BF, BF)
    got = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up)[0]
    p64.close(got, want, p64.rounded(bound, want, BF), "saturated")


def test_gradients_against_differences():
    """The gradients of sum(h * dh) in x, a scale and a bias against central
    differences of the 64-bit forward pass."""
    M, K, F, gs = 20, 128, 48, 32
    gate, up = weight(F, K, 8, gs, HF, 1), weight(F, K, 8, gs, HF, 2)
    x, dh = act(M, K, 3, HF), act(M, F, 4, HF)
    _, g, u = api.qmm_gate_up_silu(x, gate, up, save=True)
    dx, dgate, dup = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, g_dtype=F32)
    q = [p64.dequant64(w)[0] for w in (gate, up)]
    S = [w.scales.double() for w in (gate, up)]
    Z = [w.biases.double() for w in (gate, up)]
    X, D = x.double(), dh.double()

    def loss(X, S, Z):
        g, u = (X @ (q[i] * S[i].repeat_interleave(gs, 1) + Z[i].repeat_interleave(gs, 1)).t() for i in range(2))
        return float((g * torch.sigmoid(g) * u * D).sum())

    def slope(t, i, j, step):
        keep = float(t[i, j])
        at = []
        for s in (step, -step):
            t[i, j] = keep + s
            at.append(loss(X, S, Z))
        t[i, j] = keep
        return (at[0] - at[1]) / (2 * step)

    # f16 roundings of g, u, dg, du, weights and dx: 6 * 2^-11 of the magnitudes, which
    # exceed the norm's share by sqrt(terms) at most; 2% of the gradient's own scale holds them
    for t, grad in ((X, dx), (S[0], dgate[0]), (Z[0], dgate[1]), (S[1], dup[0]), (Z[1], dup[1])):
        scale = float(grad.double().square().mean().sqrt())
        for i, j in ((0, 0), (7, 1), (19, 3)):
            assert abs(slope(t, i, j, 1e-5) - float(grad[i, j])) <= 0.02 * max(scale, abs(float(grad[i, j])))


def test_other_stream_and_capture():
    M, K, F = 150, 512, 320
    gate, up = weight(F, K, 4, 64, BF, 1), weight(F, K, 4, 64, BF, 2)
    x, dh = act(M, K, 3, BF), act(M, F, 4, BF)

    def step(stream=None):
        h, g, u = api.qmm_gate_up_silu(x, gate, up, save=True, stream=stream)
        dx, dg, du = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, stream=stream)
        return [h, g, u, dx, *dg, *du, *api.qmm_matmul_backward(dh, x, gate, stream=stream)]

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x0, x1 = x.clone(), act(M, K, 99, BF)
    x.copy_(x1)
    want1 = step()
    for i, w in ((x0, want), (x1, want1), (x0, want)):
        x.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, got))


def test_wide_and_tall_weights():
    """Long sums, one column of tiles, and rows past many tiles."""
    check_matmul_backward(40, 2, 128, 16384, 70, BF, F32)
    check_forward(33, 2, 128, 16384, 70, BF)
    check_matmul_backward(20, 4, 32, 64, 20000, HF, F32)
    check_forward(150, 4, 32, 64, 20000, HF)


def test_two_streams_and_two_graphs_at_once():
    """Calls that overlap on the GPU share nothing: two streams, and two captured
    graphs replayed on two streams, give the bits of calls by themselves."""
    K, F = 1024, 640
    gate, up = weight(F, K, 4, 64, BF, 1), weight(F, K, 4, 64, BF, 2)
    sizes = (40, 300, 1700)
    data = [(act(m, K, m, BF), act(m, F, m + 1, BF)) for m in sizes]

    def step(x, dh, stream=None):
        h, g, u = api.qmm_gate_up_silu(x, gate, up, save=True, stream=stream)
        dx, dg, du = api.qmm_gate_up_silu_backward(dh, x, g, u, gate, up, stream=stream)
        return [h, g, u, dx, *dg, *du, *api.qmm_matmul_backward(dh, x, gate, stream=stream)]

    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        got = [step(*d, stream=s) for d, s in zip(data, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    graphs, outs = [], []
    for d in data:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*d))
    for o in outs:
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, outs) for a, b in zip(w, g))


def test_rows_after_the_last_token_are_left():
    """Outputs given with more memory behind them: nothing past the call's rows is
    written (odd row lengths, every path)."""
    K, F, gs = 256, 77, 32
    gate, up = weight(F, K, 6, gs, HF, 1), weight(F, K, 6, gs, HF, 2)
    for M in (1, 9, 31, 140, 600):
        x = act(M, K, M, HF)
        g = [Guarded((M, F), HF) for _ in range(3)]
        api.qmm_gate_up_silu(x, gate, up, out=g[0].out, g_pre=g[1].out, u_pre=g[2].out)
        dx = Guarded((M, K), HF)
        p = [Guarded((F, K // gs), F32) for _ in range(4)]
        api.qmm_gate_up_silu_backward(act(M, F, 5, HF), x, g[1].out, g[2].out, gate, up, dx=dx.out,
                                      dgate=(p[0].out, p[1].out), dup=(p[2].out, p[3].out))
        torch.cuda.synchronize()
        for i, t in enumerate((*g, dx, *p)):
            t.check(f"M={M} output {i}")


def test_large_scales_and_zero_weights():
    """Values at the ends of the type: weights of 1e30 in bf16, groups whose scale
    and bias are zero, and codes at both ends."""
    M, K, F, gs = 70, 128, 96, 64
    gate = weight(F, K, 4, gs, BF, 1)
    up = weight(F, K, 4, gs, BF, 2)
    gate.scales[3], gate.biases[3] = 0.0, 0.0
    gate.packed[5], gate.packed[6] = 0, -1
    up.scales[7] = 1e30
    up.biases[7] = -1e30
    x = act(M, K, 3, BF)
    (h, g, u), (eh, eg, eu) = p64.gate_up64(x, gate, up, BF)
    hh, gg, uu = api.qmm_gate_up_silu(x, gate, up, save=True)
    for got, w, e in ((gg, g, eg), (uu, u, eu)):
        err = (got.double() - w).abs()
        assert (err <= p64.rounded(e, w, BF)).all()
    err = (hh.double() - h).abs()
    assert (err <= p64.rounded(eh, h, BF)).all()
    assert (gg[:, 3] == 0).all() and (hh[:, 3] == 0).all()
    dy = act(M, F, 4, BF)
    dy[:, 7] = 0  # the row of 1e30 adds nothing
    dx, ds, dz = api.qmm_matmul_backward(dy, x, up)
    want, bound = p64.dx64([dy.double()], [up], F32, BF)
    assert torch.isfinite(dx).all() and ((dx.double() - want).abs() <= p64.rounded(bound, want, BF)).all()
    assert (ds[7] == 0).all() and (dz[7] == 0).all()


@pytest.mark.parametrize("bits,gs,K,N", [(4, 32, 512, 200), (8, 128, 2048, 150), (3, 32, 1280, 333), (6, 32, 1024, 90),
                                         (2, 64, 1024, 700), (3, 128, 2048, 70), (8, 32, 1536, 129), (2, 32, 1056, 64),
                                         (3, 32, 1440, 700), (6, 64, 1600, 257)])
@pytest.mark.parametrize("M", [50, 200])
def test_scale_windows_and_split_sums(M, bits, gs, K, N):
    """Rows of scales that come by TMA (a multiple of 8 groups) at every width and
    group size, rows of codes off 16 bytes, and sums cut over clusters."""
    check_forward(M, bits, gs, K, N, BF)
    check_matmul_backward(M, bits, gs, K, N, HF, F32)
    check_gated_backward(M, bits, gs, K, N, BF, BF)
