"""Host-side refusals of the calls on rows of logits (log probabilities,
distillation): no GPU is touched."""
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


def test_token_logprobs_arguments(lib):
    p, odd = _fake(), _fake(0x10001)

    def call(logits=p, dtype=0, stride=100, tokens=p, lens=None, N=4, R=1, V=100, K=5, logp=p, ent=p, lse=p, ti=p, tl=p):
        return lib.dspark_token_logprobs(logits, dtype, stride, tokens, lens, N, R, V, K, logp, ent, lse, ti, tl, None)

    for kw in (dict(logits=None), dict(logits=odd), dict(logits=odd, dtype=1), dict(dtype=3), dict(dtype=-1),
               dict(stride=99), dict(tokens=None), dict(N=-1), dict(R=0), dict(R=3), dict(V=0), dict(K=-1),
               dict(K=101), dict(logp=None), dict(ent=None), dict(lse=None), dict(ti=None), dict(tl=None)):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(V=(1 << 21) + 1, stride=1 << 22), dict(N=(1 << 24) + 1), dict(K=129, V=200, stride=200)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    assert call(N=0, logits=None, tokens=None, logp=None, ent=None, lse=None, ti=None, tl=None) == ds.OK


def test_emitted_logprobs_arguments(lib):
    p = _fake()

    def call(T=p, dtype=0, x=p, n=p, tok=p, B=2, gamma=4, V=100, K=0, out=p):
        return lib.dspark_emitted_logprobs(T, dtype, x, n, tok, B, gamma, V, K, out, p, p, None, None, None)

    for kw in (dict(T=None), dict(x=None), dict(n=None), dict(tok=None), dict(B=-1), dict(gamma=0), dict(K=1),
               dict(dtype=5), dict(out=None)):
        assert call(**kw) == ds.ERR_INVALID, kw
    assert call(B=65536) == ds.ERR_UNSUPPORTED and call(gamma=33) == ds.ERR_UNSUPPORTED
    assert call(B=0) == ds.OK


def test_token_logprobs_backward_arguments(lib):
    p, odd = _fake(), _fake(0x10002)

    def call(logits=p, stride=100, tokens=p, lse=p, ent=p, gl=p, gh=p, N=4, R=1, V=100, out=p):
        return lib.dspark_token_logprobs_backward(logits, 0, stride, tokens, lse, ent, gl, gh, None, N, R, V, out, None)

    for kw in (dict(logits=None), dict(tokens=None), dict(lse=None), dict(ent=None), dict(out=None), dict(out=odd),
               dict(stride=50), dict(R=3)):
        assert call(**kw) == ds.ERR_INVALID, kw
    assert call(N=0) == ds.OK


def test_distill_arguments(lib):
    p, odd = _fake(), _fake(0x10002)

    def call(logits=p, dtype=0, stride=100, ti=p, tv=p, N=4, R=2, V=100, K=5, tau=1.0, loss=p, stats=p, dl=p, gd=0):
        return lib.dspark_distill_loss(logits, dtype, stride, ti, tv, None, None, None, N, R, V, K, tau, loss, stats,
                                       dl, gd, None)

    def back(stats=p, g=p, dl=p, K=5, tau=1.0):
        return lib.dspark_distill_loss_backward(p, 0, 100, p, p, stats, g, None, None, 4, 2, 100, K, tau, dl, 0, None)

    for kw in (dict(logits=None), dict(ti=None), dict(tv=None), dict(loss=None), dict(stats=None), dict(K=0),
               dict(tau=0.0), dict(tau=-1.0), dict(tau=float("inf")), dict(tau=float("nan")), dict(tau=1e-44), dict(tau=4e-39), dict(tau=9e-31), dict(tau=1.1e30), dict(tau=3e38),
               dict(dl=odd), dict(R=3), dict(stride=99), dict(dtype=4)):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(K=129), dict(gd=2), dict(dtype=1, gd=0), dict(dtype=2, gd=1)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    assert call(N=0, R=1) == ds.OK
    for kw in (dict(stats=None), dict(g=None), dict(dl=None), dict(K=0), dict(tau=0.0)):
        assert back(**kw) == ds.ERR_INVALID, kw


def test_binding_refuses_host_tensors(lib):
    x, tok = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ds.token_logprobs(x, tok)
    with pytest.raises(ValueError):
        ds.distill_loss(x, tok[:, None], x[:, :1])


def test_head_backward_arguments(lib):
    p, odd = _fake(), _fake(0x10002)

    def call(d=p, W1=p, W2=p, wdtype=1, anchor=p, x=p, B=2, G=3, V=256, r=256, status=None, dW1=p, dW2=p, ws=p, n=1 << 30):
        return lib.dspark_markov_head_backward_ex(d, W1, W2, wdtype, anchor, x, B, G, V, r, status, dW1, dW2, ws, n, None)

    for kw in (dict(d=None), dict(W1=None), dict(W2=None), dict(anchor=None), dict(x=None), dict(dW1=None), dict(dW2=None),
               dict(d=odd), dict(W1=odd), dict(W2=odd), dict(dW1=odd), dict(dW2=odd), dict(status=odd), dict(wdtype=2),
               dict(B=0), dict(G=0), dict(V=0)):
        assert call(**kw) == ds.ERR_INVALID, kw
    for kw in (dict(wdtype=0), dict(r=128), dict(V=184), dict(V=260)):
        assert call(**kw) == ds.ERR_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=odd), dict(n=256)):
        assert call(**kw) == ds.ERR_WORKSPACE, kw
