"""Host-side refusals of the cross entropy from hidden states: no GPU is touched."""
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
