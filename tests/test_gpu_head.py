"""The Markov head's logits for given tokens and its weight gradients against
plain forms in 64 bits, and a whole training step through the public calls:
logits, distillation, head gradients."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

R = 256
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(V, seed, sigma=0.02):
    g = _gen(seed)
    return [torch.empty((V, R), device="cuda").normal_(0, sigma, generator=g).bfloat16() for _ in range(2)]


def _tokens(B, G, V, seed, most=None):
    g = _gen(seed)
    hi = V if most is None else most
    a = torch.randint(0, hi, (B,), generator=g, device="cuda", dtype=torch.int32)
    return a, torch.randint(0, hi, (B, G), generator=g, device="cuda", dtype=torch.int32)


def _prev(anchor, x):
    return torch.cat([anchor[:, None], x[:, :-1]], 1).reshape(-1).long()


SHAPES = [(1, 1, 192), (3, 2, 200), (16, 4, 4096), (128, 1, 1000), (43, 3, 2056), (65, 2, 12008), (130, 16, 5000),
          (700, 7, 264), (2, 3, 151936)]


@pytest.mark.parametrize("B,G,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_against_64_bits(B, G, V, dtype):
    W1, W2 = _weights(V, V, 0.3)
    anchor, x = _tokens(B, G, V, B)
    U = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(1))
    keep = U.clone()
    got = ds.markov_logits(U, W1, W2, anchor, x, dtype=dtype)
    assert got.dtype == dtype and torch.equal(U, keep)
    E, W = W1[_prev(anchor, x)].to(F64), W2.to(F64)
    want = U.to(F64) + (E @ W.T).view(U.shape)
    # products are exact; each of 256 additions is off by at most a step of the sum of the terms' sizes so far
    tol = 2 * ref.U * (16 + 2) * (E.abs() @ W.abs().T).view(U.shape) + 2 * ref.HALF[dtype] * want.abs()
    ref.assert_close(got, want, tol, "logits")
    if dtype == torch.float32:
        assert ds.markov_logits(U, W1, W2, anchor, x, out=U) is U
        assert torch.equal(U, got)


def _check_backward(D, W1, W2, anchor, x, ws=None):
    B, G, V = D.shape
    dW1, dW2 = ds.markov_head_backward(D, W1, W2, anchor, x, ws=ws)
    prev = _prev(anchor, x)
    ok = (prev >= 0) & (prev < V)
    d = D.reshape(B * G, V).to(F64)[ok]
    prev = prev[ok]
    E, W = W1[prev].to(F64), W2.to(F64)
    # a sum of K exact products: 16 at a time, each addition off by a step of
    # the running sum, which is at most the sum of the terms' sizes; the few
    # parts and rows of a token likewise
    def tol(size, K):
        return 2 * ref.U * (K / 16 + 20) * size
    ref.assert_close(dW2, d.T @ E, tol(d.abs().T @ E.abs(), B * G), "dW2")
    z = torch.zeros((V, R), dtype=F64, device="cuda")
    want = z.index_add(0, prev, d @ W)
    size = z.index_add(0, prev, d.abs() @ W.abs())
    ref.assert_close(dW1, want, tol(size, V + 16 * 200 + 16 * B * G), "dW1")
    used = torch.zeros(V, dtype=torch.bool, device="cuda")
    used[prev] = True
    assert (dW1[~used] == 0).all()
    return dW1, dW2


@pytest.mark.parametrize("B,G,V", SHAPES)
@pytest.mark.parametrize("most", [None, 5])
def test_backward_against_64_bits(B, G, V, most):
    W1, W2 = _weights(V, V)
    anchor, x = _tokens(B, G, V, B, most)
    D = torch.empty((B, G, V), device="cuda").normal_(0, 1, generator=_gen(2)).bfloat16()
    _check_backward(D, W1, W2, anchor, x)


def test_backward_is_near_fp32():
    # relative errors (2-norm) as an fp32 product of this length has them
    B, G, V = 128, 16, 20000
    W1, W2 = _weights(V, 1)
    anchor, x = _tokens(B, G, V, 3)
    D = torch.empty((B, G, V), device="cuda").normal_(0, 1, generator=_gen(2)).bfloat16()
    dW1, dW2 = ds.markov_head_backward(D, W1, W2, anchor, x)
    prev, d = _prev(anchor, x), D.view(-1, V).to(F64)
    w2 = d.T @ W1[prev].to(F64)
    w1 = torch.zeros((V, R), dtype=F64, device="cuda").index_add(0, prev, d @ W2.to(F64))
    for got, want in ((dW1, w1), (dW2, w2)):
        assert float((got.to(F64) - want).norm() / want.norm()) < 1e-5


def test_backward_is_reproducible():
    B, G, V = 300, 16, 1600
    W1, W2 = _weights(V, 1)
    anchor, x = _tokens(B, G, V, 3, 40)
    D = torch.empty((B, G, V), device="cuda").normal_(0, 1, generator=_gen(2)).bfloat16()
    first = ds.markov_head_backward(D, W1, W2, anchor, x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, ds.markov_head_backward(D, W1, W2, anchor, x)))


def test_tokens_out_of_range_are_reported():
    B, G, V = 5, 4, 1024
    W1, W2 = _weights(V, 1)
    anchor, x = _tokens(B, G, V, 3)
    anchor[1], x[2, 1], x[3, 0], x[4, 3] = -1, V, -7, V + 5    # (the last position's token is nobody's previous one)
    U = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(1))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = ds.markov_logits(U, W1, W2, anchor, x, ws=ws)
    assert ds.read_status(ws) == ds.ERR_INVALID
    for b, k in ((1, 0), (2, 2), (3, 1)):
        assert torch.equal(got[b, k], U[b, k])
    ws = ds.head_workspace(B, G, V, "cuda")
    _check_backward(U.bfloat16(), W1, W2, anchor, x, ws=ws)
    assert ds.read_status(ws) == ds.ERR_INVALID
    anchor, x = _tokens(B, G, V, 3)
    _check_backward(U.bfloat16(), W1, W2, anchor, x, ws=ws)
    assert ds.read_status(ws) == ds.OK


def test_logits_are_the_drafts():
    # teacher forced with its own tokens, the head gives the logits the draft
    # sampled from: their log-sum-exp and the drafted tokens' probabilities
    from speculative_decoding_02_gb300 import workloads as wl

    w = wl.custom(B=16, gamma=4, V=4096, r=256, H=64, wdtype=torch.bfloat16, u_sigma=3.0, seed=5)
    inp = wl.make_inputs(w, 0, "cuda")
    x, p, lse = ds.markov_draft(inp["U"], inp["W1"], inp["W2"], inp["anchor"], w.seed)
    l = ds.markov_logits(inp["U"], inp["W1"], inp["W2"], inp["anchor"], x)
    logp, _, got, *_ = ds.token_logprobs(l, x)
    assert (got - lse).abs().max() < 1e-4 and (logp.exp() / p - 1).abs().max() < 1e-4


@pytest.mark.parametrize("tail", [False, True])
def test_training_step(tail):
    """One step of the head's training through the public calls, against the
    same step in 64 bits, and along the gradient against differences."""
    B, G, V, K = 12, 4, 2048, 24
    W1, W2 = _weights(V, 1, 0.1)
    anchor, x = _tokens(B, G, V, 3, 50)
    U = torch.empty((B, G, V), device="cuda").normal_(0, 2, generator=_gen(1))
    T = U + torch.empty_like(U).normal_(0, 1, generator=_gen(4))
    rows = torch.randint(0, G + 1, (B,), generator=_gen(5), device="cuda", dtype=torch.int32)
    rows[0], rows[1] = 0, G
    _, _, lse, idx, lp = ds.token_logprobs(T, torch.full((B, G), -1, dtype=torch.int32, device="cuda"), top_k=K)
    tl = torch.zeros(B, G, device="cuda") if tail else None
    weight = torch.exp(-torch.arange(G, device="cuda") / G).expand(B, G).contiguous()

    l = ds.markov_logits(U, W1, W2, anchor, x)
    loss, stats, dl = ds.distill_loss(l, idx, lp, teacher_lse=tl, weight=weight, rows=rows, grad=True,
                                      grad_dtype=torch.bfloat16)
    dW1, dW2 = ds.markov_head_backward(dl, W1, W2, anchor, x)

    on = (torch.arange(G, device="cuda")[None] < rows[:, None]).reshape(-1)
    prev = _prev(anchor, x)

    def step(w1, w2):
        z = U.view(-1, V).to(F64) + w1[prev] @ w2.T
        return ref.distill(z, idx.view(-1, K), lp.view(-1, K), 1.0, None if tl is None else tl.view(-1), weight.view(-1))

    w1, w2 = W1.to(F64), W2.to(F64)
    wloss, _, wgrad, *_ = step(w1, w2)
    assert (loss.view(-1)[on] - wloss[on]).abs().max() < 1e-4 and (loss.view(-1)[~on] == 0).all()
    g = wgrad * on[:, None]
    want2 = g.T @ w1[prev]
    want1 = torch.zeros_like(w1).index_add(0, prev, g @ w2)
    # the gradient of the logits is rounded to bf16: 2^-8 of each term at most
    size2 = g.abs().T @ w1[prev].abs()
    size1 = torch.zeros_like(w1).index_add(0, prev, g.abs() @ w2.abs())
    ref.assert_close(dW2, want2, 2 ** -8 * 1.01 * size2 + 1e-6, "dW2")
    ref.assert_close(dW1, want1, 2 ** -8 * 1.01 * size1 + 1e-6, "dW1")
    # along a direction: (L(w + h d) - L(w - h d)) / 2h against the gradient's product with d
    total = lambda a, b: float((step(a, b)[0] * weight.view(-1).to(F64) * on).sum())
    for k, (w, dw, size) in enumerate(((w1, dW1, size1), (w2, dW2, size2))):
        d = torch.randn(w.shape, generator=_gen(9 + k), device="cuda", dtype=F64)
        h = 1e-5
        up, dn = [(w1 + s * h * d, w2) if k == 0 else (w1, w2 + s * h * d) for s in (1, -1)]
        diff = (total(*up) - total(*dn)) / (2 * h)
        tol = 2 ** -8 * float((size * d.abs()).sum()) + 1e-5 * (1 + abs(diff))
        assert abs(diff - float((dw.to(F64) * d).sum())) < tol


def test_a_round_feeds_training():
    """What the round verified, straight into the head's gradients: the target's
    alternatives of the verified positions as the teacher, the drafted tokens as
    the prefix; positions past a request's verify length take no part."""
    from speculative_decoding_02_gb300 import workloads as wl

    w = wl.custom(B=16, gamma=4, V=4096, r=256, H=64, wdtype=torch.bfloat16, u_sigma=3.0, seed=5, sps_b0=32.0,
                  sps_kind="steps")
    inp = wl.make_inputs(w, 0, "cuda")
    U, T, W1, W2, anchor = (inp[k] for k in ("U", "T", "W1", "W2", "anchor"))
    out = ds.round(U, T, W1, W2, inp["h"], inp["w"], anchor, seed=w.seed, sps=inp["sps"], mode=w.mode)
    B, G, V = U.shape
    none = torch.full((B, G + 1), -1, dtype=torch.int32, device="cuda")
    _, _, _, idx, lp = ds.token_logprobs(T, none, top_k=64, rows=out.ell)
    idx, lp = idx[:, :G].contiguous(), lp[:, :G].contiguous()
    l = ds.markov_logits(U, W1, W2, anchor, out.x)
    loss, stats, dl = ds.distill_loss(l, idx, lp, teacher_lse=torch.zeros(B, G, device="cuda"), rows=out.ell,
                                      grad=True, grad_dtype=torch.bfloat16)
    dW1, dW2 = ds.markov_head_backward(dl, W1, W2, anchor, out.x)
    on = (torch.arange(G, device="cuda")[None] < out.ell[:, None]).reshape(-1)
    assert on.any() and not on.all()
    z = l.view(-1, V)[on].to(F64)
    want, _, grad, size, gsize = ref.distill(z, idx.view(-1, 64)[on], lp.view(-1, 64)[on], 1.0,
                                             torch.zeros(int(on.sum()), device="cuda"), None)
    e = ref.base_error(V, 60.0) + 64 * ref.U + 4 * ref.U * 40
    ref.assert_close(loss.view(-1)[on], want, e * size, "loss")
    assert (loss.view(-1)[~on] == 0).all() and (dl.view(-1, V)[~on] == 0).all()
    prev = _prev(anchor, out.x)[on]
    w1, w2 = W1[prev].to(F64), W2.to(F64)
    tol = lambda s: 2 ** -8 * 1.01 * s + 1e-6
    ref.assert_close(dW2, grad.T @ w1, tol(grad.abs().T @ w1.abs()), "dW2")
    zero = torch.zeros((V, R), dtype=F64, device="cuda")
    ref.assert_close(dW1, zero.index_add(0, prev, grad @ w2), tol(zero.index_add(0, prev, grad.abs() @ w2.abs())), "dW1")


def test_refusals():
    B, G, V = 2, 3, 256
    W1, W2 = _weights(V, 1)
    anchor, x = _tokens(B, G, V, 3)
    U = torch.zeros((B, G, V), device="cuda")
    for bad in (dict(U=U.bfloat16()), dict(U=U[0]), dict(W2=W2.float()), dict(W1=W1[:-1]), dict(anchor=anchor[:1]),
                dict(x=x.long()), dict(x=x[:, :2]), dict(dtype=torch.float16), dict(out=U.bfloat16()),
                dict(out=U[:1])):
        with pytest.raises((ValueError, TypeError)):
            ds.markov_logits(**{"U": U, "W1": W1, "W2": W2, "anchor": anchor, "x": x, **bad})
    for w in (W1.float(), W1[:, :128].contiguous()):
        with pytest.raises(ds.DSparkError) as e:
            ds.markov_logits(U, w, w, anchor, x)
        assert e.value.code == ds.ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        ds.markov_head_backward(U, W1, W2, anchor, x)
    for ws in (torch.zeros(1024, device="cuda"), torch.zeros(1024, dtype=torch.uint8)):
        with pytest.raises((ValueError, TypeError)):
            ds.markov_logits(U, W1, W2, anchor, x, ws=ws)
    with pytest.raises(ds.DSparkError) as e:
        ds.markov_head_backward(U.bfloat16(), W1, W2, anchor, x, ws=torch.empty(512, dtype=torch.uint8, device="cuda"))
    assert e.value.code == ds.ERR_WORKSPACE
    with pytest.raises(ds.DSparkError) as e:    # V % 8
        ds.markov_logits(torch.zeros((B, G, 204), device="cuda"), W1[:204], W2[:204], anchor.clamp(max=3), x.clamp(max=3))
    assert e.value.code == ds.ERR_UNSUPPORTED


def test_streams_and_graphs():
    B, G, V = 20, 5, 6000
    data = []
    for s in range(2):
        U = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(s))
        data.append([U, *_weights(V, s), *_tokens(B, G, V, s)])

    def step(d):
        l = ds.markov_logits(*d)
        return (l, *ds.markov_head_backward(l.bfloat16(), *d[1:]))

    want = [step(d) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(step(data[k % 2]))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2]))
    static = [a.clone() for a in data[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for d, w in zip(data, want):
        for a, b in zip(static, d):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


def _bad_tokens(B, G, V):
    anchor, x = _tokens(B, G, V, 3)
    anchor[1], x[2, 1] = -1, V
    return anchor, x


def test_errors_of_logits_without_a_workspace():
    """They are kept for whoever asks, and are not a round's: its cached
    workspace for the same sizes is neither written nor made."""
    B, G, V = 6, 3, 1160
    W1, W2 = _weights(V, 1)
    anchor, x = _bad_tokens(B, G, V)
    U = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(1))
    rounds = ds.workspace(B, G, V, U.device)
    cached = len(ds._ws_cache)
    assert ds.read_status(rounds) == ds.OK
    ds.markov_logits(U, W1, W2, anchor, x)
    assert ds.read_status(rounds) == ds.OK
    status = ds.head_status("cuda")
    assert ds.read_status(status) == ds.ERR_INVALID and ds.read_status(status) == ds.OK
    good, y = _tokens(B, G, V, 3)
    ds.markov_logits(torch.zeros((B, G, V + 8), device="cuda"), *_weights(V + 8, 2), good, y)
    assert ds.read_status(ds.head_status(U.device)) == ds.OK and len(ds._ws_cache) == cached


def test_errors_of_gradients_without_a_workspace():
    B, G, V = 6, 3, 1160
    W1, W2 = _weights(V, 1)
    anchor, x = _bad_tokens(B, G, V)
    D = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(1)).bfloat16()
    status = ds.head_status("cuda")
    assert ds.read_status(status) == ds.OK
    _check_backward(D, W1, W2, anchor, x)
    assert ds.read_status(status) == ds.ERR_INVALID
    _check_backward(D, W1, W2, *_tokens(B, G, V, 3))
    assert ds.read_status(status) == ds.OK
    # a workspace of the caller's keeps its own errors
    ws = ds.head_workspace(B, G, V, "cuda")
    _check_backward(D, W1, W2, anchor, x, ws=ws)
    assert ds.read_status(status) == ds.OK and ds.read_status(ws) == ds.ERR_INVALID


@pytest.mark.parametrize("first", [False, True])
def test_captured_calls_without_a_workspace(first, monkeypatch):
    B, G, V = 6, 3, 1160
    W1, W2 = _weights(V, 1)
    anchor, x = _bad_tokens(B, G, V)
    U = torch.empty((B, G, V), device="cuda").normal_(0, 3, generator=_gen(1))
    D = U.bfloat16()
    want = (ds.markov_logits(U, W1, W2, anchor, x), *ds.markov_head_backward(D, W1, W2, anchor, x))
    ds.read_status(ds.head_status("cuda"))
    if first:   # as on a device where nothing has run before the capture
        monkeypatch.setattr(ds, "_head_status", {})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (ds.markov_logits(U, W1, W2, anchor, x), *ds.markov_head_backward(D, W1, W2, anchor, x))
    for _ in range(2):
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert ds.read_status(ds.head_status("cuda")) == (ds.OK if first else ds.ERR_INVALID)


@pytest.mark.parametrize("B,G,V", [(128, 16, 20000), (128, 16, 2048), (16, 4, 60000)])
def test_accumulators_are_promoted_in_time(B, G, V):
    """The tensor cores truncate when they add to an accumulator: half a step, or
    0.36 * 2^-23 of its value on average (1 / m over mantissas m in [1, 2) averages
    0.72), always towards zero.  After j additions of terms of no particular sign it
    is about sqrt(j) of them, so n additions lose 0.36 * 2^-23 * 2/3 n of the sum:
    9.2e-7 for the 32 of one accumulator, after which sums are rounded (1.5e-7 at
    most beside it).  Twice as many additions gave 1.3e-6."""
    W1, W2 = _weights(V, 1)
    anchor, x = _tokens(B, G, V, 3)
    D = torch.empty((B, G, V), device="cuda").normal_(0, 1, generator=_gen(2)).bfloat16()
    dW1, dW2 = ds.markov_head_backward(D, W1, W2, anchor, x)
    prev, d = _prev(anchor, x), D.view(-1, V).to(F64)
    w2 = d.T @ W1[prev].to(F64)
    w1 = torch.zeros((V, R), dtype=F64, device="cuda").index_add(0, prev, d @ W2.to(F64))
    for got, want in ((dW1, w1), (dW2, w2)):
        assert float((got.to(F64) - want).norm() / want.norm()) < 1e-6
