"""Host-side refusals of the cross entropy from hidden states and of the
orthogonalisation of an update: no GPU is touched."""
import ctypes

import pytest
import torch

import speculative_decoding_02_gb300 as ds


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_02_gb300 import build

    build.build()
    return ds.library()


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


BIG = 1 << 50


def test_loss_arguments(lib):
    p, odd = _fake(), _fake(0x10001)

    def call(h=p, hs=64, W=p, Ws=64, dtype=1, tokens=p, lens=None, N=6, R=2, V=100, D=64, loss=p, lse=p, status=None,
             ws=p, n=BIG):
        return lib.dspark_linear_cross_entropy(h, hs, W, Ws, dtype, tokens, lens, N, R, V, D, loss, lse, status, ws, n, None)

    for kw in (dict(h=None), dict(h=odd), dict(W=None), dict(W=_fake(0x10008)), dict(tokens=None), dict(loss=None),
               dict(lse=None), dict(status=_fake(0x10002)), dict(dtype=3), dict(dtype=-1), dict(hs=63), dict(Ws=56),
               dict(Ws=68), dict(N=-1), dict(R=0), dict(R=4), dict(V=0), dict(D=0), dict(Ws=1 << 40)):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(dtype=0), dict(N=(1 << 20) + 2), dict(V=(1 << 21) + 1), dict(D=60), dict(D=16392, hs=20000, Ws=20000)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=_fake(0x10010)), dict(n=256)):
        assert call(**kw) == ds.ERR_WORKSPACE, kw
    assert call(n=lib.dspark_linear_ce_workspace_size(6, 100, 64, 0) - 1) == ds.ERR_WORKSPACE
    assert call(N=0, h=None, W=None, tokens=None, loss=None, lse=None, ws=None) == ds.OK


def test_backward_arguments(lib):
    p, odd = _fake(), _fake(0x10008)

    def call(h=p, W=p, dtype=2, lse=p, g=p, gl=None, N=6, R=2, V=100, D=64, dh=p, dW=p, status=None, ws=p, n=BIG):
        return lib.dspark_linear_cross_entropy_backward(h, 64, W, 64, dtype, p, None, lse, g, gl, N, R, V, D, dh, dW,
                                                        status, ws, n, None)

    for kw in (dict(h=None), dict(W=None), dict(lse=None), dict(g=None), dict(dh=odd), dict(dW=odd), dict(dh=None, dW=None),
               dict(status=_fake(0x10002)), dict(dtype=9)):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(dtype=0), dict(D=4096 + 4)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(n=256), dict(n=lib.dspark_linear_ce_workspace_size(6, 100, 64, 1) - 1)):
        assert call(**kw) == ds.ERR_WORKSPACE, kw
    assert call(N=0, dW=None) == ds.OK


def test_workspace_sizes(lib):
    size = lib.dspark_linear_ce_workspace_size
    for a in ((0, 100, 64, 0), (6, 0, 64, 0), (6, 100, 0, 0), (6, 100, 60, 0), (6, 100, 64, 4), (6, 100, 64, -1),
              ((1 << 20) + 1, 100, 64, 0), (6, (1 << 21) + 1, 64, 0), (6, 100, 16392, 3)):
        assert size(*a) == 0, a
    # the largest sizes: no overflow, and the slopes of a piece stay within their bound
    big = size(1 << 20, 1 << 21, 16384, 3)
    rows = 1 << 20
    assert big > 2 * rows * 16384 + 4 * rows * 16384 + 2 * 256 * rows
    assert big < 2 * rows * 16384 + 4 * rows * 16384 + 2 * 256 * rows + 64 * rows
    assert size(2048, 151936, 2560, 3) < (256 + 2 * 256 + 32) << 20


def test_binding_refuses_host_tensors(lib):
    h, W, t = torch.zeros(2, 8).bfloat16(), torch.zeros(9, 8).bfloat16(), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ds.linear_cross_entropy(h, W, t)
    with pytest.raises(ValueError):
        ds.linear_cross_entropy_backward(h, W, t, torch.zeros(2), torch.zeros(2))


def test_newton_schulz_arguments(lib):
    p = _fake()

    def call(M=p, dtype=0, stride=30, rows=20, cols=30, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, out=p, status=None, ws=p,
             n=BIG):
        return lib.dspark_newton_schulz(M, dtype, stride, rows, cols, steps, a, b, c, eps, out, status, ws, n, None)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(M=None), dict(M=_fake(0x10002)), dict(out=None), dict(out=_fake(0x10001)), dict(dtype=3), dict(dtype=-1),
               dict(stride=29), dict(rows=-1), dict(cols=-1), dict(steps=0), dict(a=nan), dict(b=inf), dict(c=-inf),
               dict(eps=-1e-9), dict(eps=nan), dict(eps=inf), dict(status=_fake(0x10002))):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(rows=16385, cols=16385, stride=20000), dict(cols=(1 << 21) + 1, stride=1 << 22), dict(steps=65)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=_fake(0x10080)), dict(n=lib.dspark_newton_schulz_workspace_size(20, 30) - 1)):
        assert call(**kw) == ds.ERR_WORKSPACE, kw
    assert call(rows=0, M=None, out=None, ws=None) == ds.OK and call(cols=0, stride=0) == ds.OK
    size = lib.dspark_newton_schulz_workspace_size
    assert size(0, 4) == 0 and size(4, 0) == 0 and size(16385, 16385) == 0 and size(1, (1 << 21) + 1) == 0
    # the largest: no overflow
    assert 8 * 16384 * (1 << 21) < size(16384, 1 << 21) < (8 * 16384 * (1 << 21)) * 1.1


def test_newton_schulz_refuses_host_tensors(lib):
    with pytest.raises(ValueError):
        ds.newton_schulz(torch.zeros(4, 4))
