"""Refusals of the embedding, gated projection and gradient calls, without a
GPU: the C ABI's host checks and the binding's."""
import ctypes

import pytest
import torch

from weight_only_quantized_qmm_b200 import _lib, api

A = 0x10000  # an aligned fake device address: never dereferenced by these calls
BF, HF, F32 = _lib.QMM_BF16, _lib.QMM_F16, _lib.QMM_F32


@pytest.fixture(scope="module")
def L():
    return _lib.load()


def qw(bits=4, gs=64, rows=8, cols=128, sdtype=BF, mode=0, packed=A):
    return _lib.QWeightC(packed, A, A, sdtype, rows, cols, gs, bits, mode)


def mx():
    return qw(mode=_lib.QMM_MODE_MXFP4, sdtype=_lib.QMM_U8, bits=4, gs=32)


def test_embedding(L):
    def call(w=None, ids=A, n=4, out=A, out_dtype=BF, status=None):
        w = w or qw()
        return L.qmm_embedding(ids, n, ctypes.byref(w), 1.0, out, out_dtype, status, None)

    assert call(n=0) == _lib.QMM_OK
    assert call(n=-1) == call(n=2 ** 31) == _lib.QMM_ERR_INVALID_ARG
    assert call(w=qw(bits=5)) == call(w=qw(gs=48)) == _lib.QMM_ERR_INVALID_ARG
    assert call(out_dtype=9) == _lib.QMM_ERR_DTYPE
    assert call(ids=0) == call(ids=A + 2) == call(out=A + 8) == call(status=A + 1) == _lib.QMM_ERR_ALIGNMENT
    assert call(w=qw(packed=A + 4)) == _lib.QMM_ERR_ALIGNMENT
    assert call(w=qw(mode=7)) == _lib.QMM_ERR_UNSUPPORTED
    assert call(w=mx(), n=0) == _lib.QMM_OK


def test_embedding_backward(L):
    need = L.qmm_embedding_backward_workspace_bytes
    assert need(10, 100, 128) >= 0 and need(0, 0, 32) >= 0
    assert need(-1, 100, 128) == need(10, -1, 128) == need(10, 100, 0) == need(2 ** 31, 1, 32) == -1

    def call(w=None, dy=A, dy_dtype=BF, ids=A, n=4000, ds=A, dz=A, g=BF, ws=A, nb=1 << 40, status=None):
        w = w or qw()
        return L.qmm_embedding_backward(dy, dy_dtype, ids, n, ctypes.byref(w), 1.0, ds, dz, g, ws, nb, status, None)

    assert call(n=-1) == call(nb=0) == call(w=qw(bits=1)) == _lib.QMM_ERR_INVALID_ARG
    assert call(w=mx()) == _lib.QMM_ERR_UNSUPPORTED
    assert call(dy_dtype=3) == call(g=4) == _lib.QMM_ERR_DTYPE
    for bad in (dict(dy=A + 2), dict(ids=A + 1), dict(ds=0), dict(dz=A + 4), dict(ws=A + 8), dict(status=A + 3)):
        assert call(**bad) == _lib.QMM_ERR_ALIGNMENT, bad


def test_gate_up(L):
    def call(g=None, u=None, x=A, xt=BF, M=2, K=128, h=A, ht=BF, gp=None, up=None, ws=A, nb=1 << 40):
        g, u = g or qw(), u or qw()
        return L.qmm_gate_up_silu(x, xt, M, K, ctypes.byref(g), ctypes.byref(u), h, ht, gp, up, ws, nb, None)

    assert call(M=0) == _lib.QMM_OK
    assert call(M=-1) == call(K=64) == call(gp=A) == call(up=A) == _lib.QMM_ERR_INVALID_ARG
    odd = dict(g=qw(bits=3, gs=32, cols=96), u=qw(bits=3, gs=32, cols=96), M=17, K=96)  # needs its workspace
    assert call(**odd, nb=0) == _lib.QMM_ERR_INVALID_ARG
    for other in (qw(rows=16), qw(bits=8), qw(gs=32), qw(cols=64)):
        assert call(u=other) == _lib.QMM_ERR_INVALID_ARG
    assert call(xt=HF) == call(ht=HF) == call(u=qw(sdtype=HF)) == _lib.QMM_ERR_DTYPE
    f = qw(sdtype=F32)
    assert call(f, f, xt=F32, ht=F32) == call(mx(), mx()) == call(M=2 ** 31) == _lib.QMM_ERR_UNSUPPORTED
    for bad in (dict(x=A + 2), dict(h=A + 8), dict(x=0), dict(odd, ws=A + 2), dict(odd, ws=None),
                dict(gp=A + 2, up=A), dict(gp=A, up=A + 2)):
        assert call(**bad) == _lib.QMM_ERR_ALIGNMENT, bad


def test_backward(L):
    for need in (L.qmm_matmul_backward_workspace_bytes, L.qmm_gate_up_silu_backward_workspace_bytes,
                 L.qmm_gate_up_silu_workspace_bytes):
        assert need(0, 32, 0, 4) >= 0 and need(100, 128, 77, 3) >= 0
        assert need(-1, 128, 8, 4) == need(8, 2 ** 31, 8, 4) == need(8, 128, -1, 4) == need(8, 33, 8, 3) == -1

    def one(w=None, dy=A, x=A, xt=BF, M=2, K=128, dx=A, ds=A, dz=A, g=BF, ws=A, nb=1 << 40):
        w = w or qw()
        return L.qmm_matmul_backward(dy, x, xt, M, K, ctypes.byref(w), dx, ds, dz, g, ws, nb, None)

    def two(w=None, dy=A, x=A, xt=BF, M=2, K=128, dx=A, ds=A, dz=A, g=BF, ws=A, nb=1 << 40, u=None):
        w = w or qw()
        u = u or w
        return L.qmm_gate_up_silu_backward(dy, x, A, A, xt, M, K, ctypes.byref(w), ctypes.byref(u), dx, ds, dz,
                                           ds, dz, g, ws, nb, None)

    for call in (one, two):
        for bad in (dict(M=-1), dict(K=64), dict(w=qw(rows=9), nb=0), dict(dx=None, ds=None, dz=None), dict(ds=None),
                    dict(dz=None), dict(w=qw(bits=7))):
            assert call(**bad) == _lib.QMM_ERR_INVALID_ARG, bad
        for bad in (dict(xt=HF), dict(g=HF), dict(g=5)):
            assert call(**bad) == _lib.QMM_ERR_DTYPE, bad
        for bad in (dict(w=mx()), dict(w=qw(sdtype=F32), xt=F32, g=F32)):
            assert call(**bad) == _lib.QMM_ERR_UNSUPPORTED, bad
        for bad in (dict(dy=A + 2), dict(x=A + 4), dict(dx=A + 8), dict(ds=A + 2), dict(dz=A + 2), dict(w=qw(rows=9), ws=A + 4),
                    dict(w=qw(rows=9), ws=None), dict(w=qw(packed=0))):
            assert call(**bad) == _lib.QMM_ERR_ALIGNMENT, bad
    assert two(u=qw(rows=9)) == two(u=qw(bits=8)) == _lib.QMM_ERR_INVALID_ARG


def test_status_text():
    assert "token" in _lib.status_string(_lib.QMM_ERR_BAD_TOKEN_ID)


# ---------------------------------------------------------------- the binding
def host(rows=32, cols=128, bits=4, gs=64):
    z = torch.zeros(rows, cols // gs, dtype=torch.bfloat16)
    return api.QWeight(torch.zeros(rows, cols * bits // 32, dtype=torch.int32), z, z.clone(), rows, cols, gs, bits)


def refuses(match, fn):
    with pytest.raises((ValueError, _lib.QmmError), match=match):
        fn()


def test_binding():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    ids, w = z(4, t=torch.int32), host()
    refuses("CUDA", lambda: api.qmm_embedding(ids, w))
    refuses("dtype", lambda: api.qmm_embedding(ids.long(), w))
    refuses("contiguous", lambda: api.qmm_embedding(z(8, t=torch.int32)[::2], w))
    refuses("expected", lambda: api.qmm_embedding(ids, w, out=z(5, 128)))
    refuses("out has shape", lambda: api.qmm_embedding(ids, w, out=z(3, 128)))
    refuses("CUDA", lambda: api.qmm_embedding_backward(z(4, 128), ids, w))
    refuses("dy has shape", lambda: api.qmm_embedding_backward(z(3, 128), ids, w))
    refuses("dscales", lambda: api.qmm_embedding_backward(z(4, 128), ids, w, dscales=z(31, 2)))
    refuses("dtype", lambda: api.qmm_embedding_backward(z(4, 128), ids, w, dscales=z(32, 2), g_dtype=torch.float32))
    refuses("workspace", lambda: api.qmm_embedding_backward(z(4000, 128), z(4000, t=torch.int32), w,
                                                            workspace=z(1, t=torch.uint8)))
    x, dh = z(3, 128), z(3, 32)
    refuses("CUDA", lambda: api.qmm_gate_up_silu(x, w, w))
    refuses("out has shape", lambda: api.qmm_gate_up_silu(x, w, w, out=z(2, 32)))
    refuses("g_pre has dtype", lambda: api.qmm_gate_up_silu(x, w, w, g_pre=z(3, 32, t=torch.float32)))
    refuses("CUDA", lambda: api.qmm_matmul_backward(dh, x, w))
    refuses("dy has shape", lambda: api.qmm_matmul_backward(z(3, 31), x, w))
    refuses("dy has dtype", lambda: api.qmm_matmul_backward(dh.float(), x, w))
    refuses("invalid argument", lambda: api.qmm_matmul_backward(dh, z(3, 64), w))
    refuses("dx", lambda: api.qmm_matmul_backward(dh, x, w, dx=z(3, 64)))
    refuses("CUDA", lambda: api.qmm_gate_up_silu_backward(dh, x, dh, dh, w, w))
    refuses("u_pre has shape", lambda: api.qmm_gate_up_silu_backward(dh, x, dh, z(3, 16), w, w))
    refuses("invalid argument", lambda: api.qmm_gate_up_silu_backward(dh, x, dh, dh, w, host(rows=16)))
    refuses("dup_scales", lambda: api.qmm_gate_up_silu_backward(dh, x, dh, dh, w, w, dup=(z(1, 2), z(32, 2))))
    small = host()
    small.scales = small.scales[:31]
    refuses("gate: qmm: scales holds", lambda: api.qmm_gate_up_silu(x, small, w))


def test_largest_sizes(L):
    """Rows and columns past the last one of a tile are counted in 32 bits too."""
    most = 2 ** 31 - 1024
    for need in (L.qmm_matmul_backward_workspace_bytes, L.qmm_gate_up_silu_backward_workspace_bytes,
                 L.qmm_gate_up_silu_workspace_bytes):
        assert need(most, 32, 8, 4) >= 0 and need(8, most, 8, 4) >= 0 and need(8, 32, most, 4) >= 0
        assert need(most + 1, 32, 8, 4) == need(8, most + 32, 8, 4) == need(8, 32, most + 1, 4) == -1

    def gate_up(M, rows):
        g = u = qw(rows=rows)
        return L.qmm_gate_up_silu(A, BF, M, 128, ctypes.byref(g), ctypes.byref(u), A, BF, None, None, A, 1 << 60, None)

    def matmul(M, rows):
        w = qw(rows=rows)
        return L.qmm_matmul_backward(A, A, BF, M, 128, ctypes.byref(w), A, A, A, BF, A, 1 << 60, None)

    for call in (gate_up, matmul):
        assert call(most + 1, 8) == call(2 ** 31 - 1, 8) == call(20, most + 1) == _lib.QMM_ERR_UNSUPPORTED
    need = L.qmm_embedding_backward_workspace_bytes
    assert need(10, 2 ** 30, 32) >= 0 and need(10, 2 ** 30 + 1, 32) == need(10, 2 ** 31 - 2, 32) == -1
    w = qw(rows=2 ** 31 - 2)
    assert L.qmm_embedding_backward(A, BF, A, 10, ctypes.byref(w), 1.0, A, A, BF, A, 1 << 60, None,
                                    None) == _lib.QMM_ERR_INVALID_ARG
