"""The lookup in a packed table and the gradient of its scales and biases,
against 64-bit forms."""
import pytest
import torch

from tests import plain64 as p64
from tests.helpers import Guarded
from weight_only_quantized_qmm_b200 import _lib, api
from weight_only_quantized_qmm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def table(rows, cols, bits, gs, dtype=torch.bfloat16, seed=1):
    return api.qmm_quantize(wl.gen_weight(rows, cols, seed).to(DEV), gs, bits, dtype)


def some_ids(n, rows, seed=2):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, rows, (n,), generator=g, dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("bits,gs,cols", [(2, 32, 32), (3, 32, 96), (3, 64, 320), (4, 64, 4096), (4, 128, 128),
                                          (6, 32, 2080), (6, 128, 1280), (8, 64, 64)])
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                       (torch.float32, torch.float16)])
def test_lookup(bits, gs, cols, dtype, out):
    rows, alpha = 301, 7.25
    qw = table(rows, cols, bits, gs, dtype)
    _, W = p64.dequant64(qw)
    for n in (1, 2, 77):
        ids = some_ids(n, rows)
        ids[-1] = rows - 1
        g = Guarded((n, cols), out)
        api.qmm_embedding(ids, qw, alpha, out=g.out)
        want = W[ids.long()] * alpha
        # the dequantized value and the product: one fp32 rounding each
        bound = 2 * p64.U[torch.float32] * want.abs() + 1e-40
        p64.close(g.check(), want, p64.rounded(bound, want, out), f"lookup n={n}")


def test_lookup_equals_dequantize_rows():
    for mode, (bits, gs) in api.MX_PARAMS.items():
        rows, cols = 50, 160
        g = torch.Generator().manual_seed(mode)
        packed = torch.randint(-2 ** 31, 2 ** 31, (rows, cols * bits // 32), generator=g).to(torch.int32).to(DEV)
        scales = torch.randint(100, 140, (rows, cols // gs), generator=g).to(torch.uint8).to(DEV)
        qw = api.mx_qweight(packed, scales, mode, rows, cols)
        ids = some_ids(33, rows).view(3, 11)
        for out in (torch.float32, torch.bfloat16):
            want = api.qmm_dequantize(qw, out)[ids.long()]
            assert torch.equal(api.qmm_embedding(ids, qw, y_dtype=out), want)
    qw = table(64, 256, 4, 64)
    ids = some_ids(20, 64)
    assert torch.equal(api.qmm_embedding(ids, qw), api.qmm_dequantize(qw, torch.bfloat16)[ids.long()])


def test_lookup_bad_ids_and_no_tokens():
    qw = table(40, 128, 4, 64)
    ids = torch.tensor([3, -1, 40, 39, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = api.qmm_embedding(ids, qw, 2.0, torch.float32, d_status=status)
    assert int(status) == _lib.QMM_ERR_BAD_TOKEN_ID
    bad = torch.tensor([False, True, True, False, True, True, False], device=DEV)
    assert (y[bad] == 0).all()
    assert torch.equal(y[~bad], 2.0 * api.qmm_dequantize(qw)[ids[~bad].long()])
    status.zero_()
    api.qmm_embedding(ids[~bad].contiguous(), qw, d_status=status)
    assert int(status) == 0
    assert api.qmm_embedding(ids[:0], qw).shape == (0, 128)


def grad64(dy, ids, qw, alpha):
    q, _ = p64.dequant64(qw)
    a = torch.zeros(qw.rows, qw.cols, dtype=torch.float64, device=DEV)
    mag = a.clone()
    ok = (ids >= 0) & (ids < qw.rows)
    a.index_add_(0, ids[ok].long(), dy.double()[ok] * alpha)
    mag.index_add_(0, ids[ok].long(), dy.double()[ok].abs() * abs(alpha))
    count = torch.zeros(qw.rows, dtype=torch.float64, device=DEV).index_add_(
        0, ids[ok].long(), torch.ones(int(ok.sum()), dtype=torch.float64, device=DEV))
    # fp32 sums of `count` tokens, then of a group's products: one rounding each
    bound = mag * (count + qw.group_size + 4).unsqueeze(1) * 2.0 ** -24
    gs = qw.group_size
    return ((p64.by_group(a * q, gs), p64.by_group(a, gs)), (p64.by_group(bound * q, gs), p64.by_group(bound, gs)))


def check_grad(dy, ids, qw, alpha, g_dtype, what):
    G = qw.cols // qw.group_size
    gs_, gb = Guarded((qw.rows, G), g_dtype), Guarded((qw.rows, G), g_dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.qmm_embedding_backward(dy, ids, qw, alpha, dscales=gs_.out, dbiases=gb.out, d_status=status)
    want, bound = grad64(dy.reshape(-1, qw.cols), ids.reshape(-1), qw, alpha)
    for got, w, b, n in zip((gs_, gb), want, bound, ("scales", "biases")):
        p64.close(got.check(f"{what} {n}"), w, p64.rounded(b, w, g_dtype), f"{what} {n}")
    return int(status)


@pytest.mark.parametrize("bits,gs,cols", [(2, 32, 32), (3, 32, 96), (3, 128, 384), (4, 64, 4096), (4, 32, 2080),
                                          (6, 64, 320), (8, 128, 1280)])
@pytest.mark.parametrize("dy_type,g_dtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                             (torch.float32, torch.float16)])
def test_gradient(bits, gs, cols, dy_type, g_dtype):
    rows = 203
    qw = table(rows, cols, bits, gs, torch.float16)
    for n, spread in ((1, rows), (2, 1), (100, 7), (333, rows)):
        dy = wl.gen_x(n, cols, 5).to(dy_type).to(DEV) * 0.05
        assert check_grad(dy, some_ids(n, spread, n), qw, 3.5, g_dtype, f"n={n}") == 0


@pytest.mark.parametrize("n,rows,kind", [(512, 90000, "spread"), (512, 3, "few"), (500, 77, "one"), (511, 40, "skewed"),
                                         (513, 90000, "spread"), (1500, 40, "skewed"), (2048, 1, "single row"),
                                         (5000, 70000, "spread"), (4097, 3, "few"), (3000, 1000, "one"),
                                         (20000, 500, "skewed"), (2049, 1, "single row")])
def test_gradient_long(n, rows, kind):
    cols = 256
    qw = table(rows, cols, 4, 64)
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(0, rows, (n,), generator=g)
    if kind == "one":
        ids[:] = 7
    if kind == "skewed":
        ids = (torch.rand(n, generator=g) ** 8 * rows).long().clamp_(0, rows - 1)
    dy = wl.gen_x(n, cols, 6).to(DEV) * 0.01
    ids = ids.to(torch.int32).to(DEV)
    assert check_grad(dy, ids, qw, 1.0, torch.float32, kind) == 0
    # the same call gives the same bits
    a, b = (api.qmm_embedding_backward(dy, ids, qw, g_dtype=torch.float32) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_bad_ids_and_no_tokens():
    qw = table(30, 128, 4, 64)
    dy = wl.gen_x(6, 128, 3).to(DEV)
    ids = torch.tensor([3, -1, 30, 3, -2 ** 31, 29], dtype=torch.int32, device=DEV)
    assert check_grad(dy, ids, qw, 1.0, torch.float32, "bad ids") == _lib.QMM_ERR_BAD_TOKEN_ID
    assert check_grad(dy[:0], ids[:0], qw, 1.0, torch.float32, "no tokens") == 0
    # a NaN gradient of a token without a row goes nowhere
    dy2 = dy.clone()
    dy2[1] = float("nan")
    for a, b in zip(api.qmm_embedding_backward(dy, ids, qw), api.qmm_embedding_backward(dy2, ids, qw)):
        assert torch.equal(a, b)


def test_gradient_is_the_slope_of_the_lookup():
    """Against differences: the lookup is linear in scales and biases, so a
    step in one of them moves sum(y * dy) by the gradient times the step."""
    rows, cols, gs = 12, 128, 64
    qw = table(rows, cols, 4, gs, torch.float32)
    ids = some_ids(40, rows)
    dy = wl.gen_x(40, cols, 9, "f32").to(DEV)
    ds, dz = api.qmm_embedding_backward(dy, ids, qw, 2.0)
    loss = lambda: float((api.qmm_embedding(ids, qw, 2.0).double() * dy.double()).sum())  # noqa: E731
    for t, grad in ((qw.scales, ds), (qw.biases, dz)):
        for r, g in ((0, 0), (5, 1), (11, 0)):
            keep = float(t[r, g])
            at = []
            for step in (0.5, -0.5):
                t[r, g] = keep + step
                at.append(loss())
            t[r, g] = keep
            # values to 64 * 15 * 0.5 * 2, each output off by 2 roundings of fp32, 40 * 128 of them
            assert abs((at[0] - at[1]) - float(grad[r, g])) <= 1e-3 * max(1.0, abs(float(grad[r, g])))


def test_other_stream_and_capture():
    qw = table(500, 512, 4, 64)
    ids, dy = some_ids(700, 500), wl.gen_x(700, 512, 4).to(DEV)
    want = (api.qmm_embedding(ids, qw, 2.0), *api.qmm_embedding_backward(dy, ids, qw, 2.0))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (api.qmm_embedding(ids, qw, 2.0, stream=s), *api.qmm_embedding_backward(dy, ids, qw, 2.0, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (api.qmm_embedding(ids, qw, 2.0), *api.qmm_embedding_backward(dy, ids, qw, 2.0))
    ids2 = some_ids(700, 500, 77)
    want2 = (api.qmm_embedding(ids2, qw, 2.0), *api.qmm_embedding_backward(dy, ids2, qw, 2.0))
    for i, w in ((ids.clone(), want), (ids2, want2), (ids.clone(), want)):
        ids.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, got))


def test_offsets_past_32_bits():
    """A table of 9.8 GB: rows whose codes start past 2^32 bytes, and whose dense
    index passes 2^33."""
    rows, cols, gs = 600_000, 16384, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    packed = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols // 4), dtype=torch.int32, device=DEV, generator=g)
    scales = torch.rand(rows, cols // gs, device=DEV, generator=g).to(torch.bfloat16)
    qw = api.QWeight(packed, scales, -scales, rows, cols, gs, 8)
    ids = torch.tensor([rows - 1, 0, 599_123, rows - 1, 262_144, 300_001], dtype=torch.int32, device=DEV)
    u, where = torch.unique(ids.long(), return_inverse=True)
    small = api.QWeight(packed[u].contiguous(), scales[u].contiguous(), -scales[u].contiguous(), u.numel(), cols, gs, 8)
    _, W = p64.dequant64(small)
    want = W[where] * 2.0
    bound = 2 * p64.U[torch.float32] * want.abs()
    p64.close(api.qmm_embedding(ids, qw, 2.0, torch.float32), want, p64.rounded(bound, want, torch.float32), "lookup")
    for n in (ids.numel(), 900):  # both ways the list is taken
        many = ids.repeat(-(-n // ids.numel()))[:n].contiguous()
        dy = (wl.gen_x(n, 512, 4).to(DEV) * 0.1).repeat(1, cols // 512)
        ds, dz = api.qmm_embedding_backward(dy, many, qw, 2.0, g_dtype=torch.float32)
        w = where.repeat(-(-n // ids.numel()))[:n].to(torch.int32)
        wants, bounds = grad64(dy, w, small, 2.0)
        for got, wt, b in zip((ds, dz), wants, bounds):
            p64.close(got[u], wt, p64.rounded(b, wt, torch.float32), f"gradient n={n}")
            assert int((got.abs().sum(1) > 0).sum()) == u.numel()
