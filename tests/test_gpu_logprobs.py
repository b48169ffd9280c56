"""Log probabilities of given tokens, the rows' entropies and their top
alternatives, and the gradient of the first two, against plain forms in 64 bits:
types, odd sizes and strides, ragged rows, masked and empty rows, ties, NaN and
infinities, refusals, streams and graphs."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
LOWEST = {d: torch.finfo(d).min for d in DTYPES}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def _tokens(N, V, seed):
    return torch.randint(0, V, (N,), dtype=torch.int32, device="cuda",
                         generator=torch.Generator(device="cuda").manual_seed(seed))


def _check(x, tokens, K, got=None):
    got = ds.token_logprobs(x, tokens, top_k=K) if got is None else got
    want = ref.logprobs(x, tokens, K)
    z = x.to(ref.F64)
    fin = torch.where(z > -3e38, z, torch.full_like(z, math.nan))
    # the entries with weight lie at most 104 + log V below the largest (below
    # that exp is 0 in float32), so only so much of a row's span counts
    span = min(120.0, float(torch.nan_to_num(fin.nan_to_num(-math.inf).amax(-1) - fin.nan_to_num(math.inf).amin(-1),
                                             nan=0.0, posinf=0.0, neginf=0.0).max()))
    e = ref.base_error(x.shape[-1], span)
    lse = want[2].abs().nan_to_num(posinf=0.0)
    step = 2 * ref.U
    ref.assert_close(got[2], want[2], e + step * lse, "lse")
    lp = want[0].abs().nan_to_num(posinf=0.0)
    ref.assert_close(got[0], want[0], e + step * (lse + lp + 8), "logp")
    H = want[1]
    ref.assert_close(got[1], H, e * (3 + 2 * H), "entropy")
    if K == 0:
        assert got[3] is None and got[4] is None
        return
    assert torch.equal(got[3], want[3]), "alternatives"
    tl = want[4].abs().nan_to_num(posinf=0.0)
    ref.assert_close(got[4], want[4], e + step * (lse[:, None] + tl + 8), "top_logp")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (2, 7, 0), (5, 31, 31), (4, 1000, 20), (7, 4099, 128),
                                   (1, 151936, 20), (9, 50257, 64), (330, 2053, 5), (3, 262144, 128), (2, 300001, 1),
                                   (1, 2097152, 33)])
def test_against_64_bits(dtype, N, V, K):
    _check(ref.logits(N, V, dtype, 7 * N + V), _tokens(N, V, V), K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V,K", [(1300, 3, 1), (1301, 41, 3), (1300, 1037, 20), (2000, 4097, 0)])
def test_more_rows_than_run_at_once(dtype, N, V, K):
    _check(ref.logits(N, V, dtype, N), _tokens(N, V, V), K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off,pad", [(1, 0), (3, 5), (0, 1), (7, 9)])
def test_strided_rows(dtype, off, pad):
    N, V = 6, 1500 + pad
    buf = ref.logits(N, V + off + pad, dtype, 3)
    x = buf[:, off:off + V]
    _check(x, _tokens(N, V, 1), 17)
    whole = buf.clone()
    g = torch.randn(N, device="cuda")
    out = ds.token_logprobs_backward(x, _tokens(N, V, 1), ds.token_logprobs(x, _tokens(N, V, 1))[2], g_logp=g)
    assert out.is_contiguous() and torch.equal(buf, whole)
    want, _ = ref.logprobs_backward(x, _tokens(N, V, 1), ds.token_logprobs(x, _tokens(N, V, 1))[2],
                                    torch.zeros(N, device="cuda"), g, torch.zeros(N, device="cuda"))
    ref.assert_close(out, want, ref.HALF[dtype] * want.abs() + 2 ** -18 * want.abs() + ref.TINY[dtype], "gradient")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [5, 1024, 20011])
def test_masked_and_empty_rows(dtype, V):
    x = ref.logits(8, V, dtype, V)
    x[0] = -math.inf                      # nothing left
    x[1] = LOWEST[dtype]                  # the type's lowest everywhere: uniform
    x[2] = -math.inf; x[2, V // 2] = 3.0  # one entry left
    x[3, ::2] = -math.inf
    x[4, 1:] = LOWEST[dtype]
    x[5] = 0.25                           # all equal
    x[6, : V - 1] = -math.inf
    x[7] = -0.0; x[7, V // 3] = 0.0       # zeros of both signs are equal
    tok = torch.tensor([0, V - 1, V // 2, 0, 0, V // 3, V - 1, V - 1], dtype=torch.int32, device="cuda")
    K = min(V, 20)
    _check(x, tok, K)
    logp, H, lse, idx, top = ds.token_logprobs(x, tok, top_k=K)
    assert lse[0] == -math.inf and logp[0] == -math.inf and H[0] == 0 and (idx[0] == -1).all()
    assert idx[5].tolist() == list(range(K)) and idx[7].tolist() == list(range(K))
    assert logp[3] == -math.inf and H[2] == 0 and logp[2] == 0
    g = ds.token_logprobs_backward(x, tok, lse, H, torch.ones(8, device="cuda"), torch.ones(8, device="cuda"))
    assert torch.isfinite(g.float()).all() and (g[0] == 0).all()
    want, size = ref.logprobs_backward(x, tok, lse, H, torch.ones(8, device="cuda"), torch.ones(8, device="cuda"))
    # (lse up to 1024 in size is rounded, which moves p by half a step of it)
    tol = (4 + lse.double().abs().clamp(max=1024.0)[:, None]) * ref.U * size + (V / 512 + 64) * ref.U * size
    ref.assert_close(g, want, tol + 2 * ref.HALF[dtype] * want.abs() + ref.TINY[dtype], "gradient")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["ascending", "descending", "steps", "one block", "equal"])
@pytest.mark.parametrize("V,K,N", [(20000, 128, 2), (151936, 64, 1), (151936, 20, 400)])
def test_alternatives_of_ordered_and_tied_rows(dtype, kind, V, K, N):
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"ascending": i / V * 9, "descending": -i / V * 9, "steps": (i // 977) % 7,
           "one block": (i < 2000).float() * 5 + i.remainder(13) * 0.01, "equal": i * 0}[kind].to(dtype)
    x = row.expand(N, V).contiguous()
    got = ds.token_logprobs(x, torch.zeros(N, dtype=torch.int32, device="cuda"), top_k=K)
    want = torch.sort(row.float(), descending=True, stable=True).indices[:K].to(torch.int32)
    assert torch.equal(got[3], want.expand(N, K))


def test_nan_and_inf_rows_are_reported():
    x = ref.logits(5, 3001, torch.float32, 5)
    want = ds.token_logprobs(x, _tokens(5, 3001, 2), top_k=4)
    y = x.clone()
    y[1, 2999] = math.nan
    y[3, 7] = math.inf
    got = ds.token_logprobs(y, _tokens(5, 3001, 2), top_k=4)
    for g, w in zip(got, want):
        assert torch.equal(g[[0, 2, 4]], w[[0, 2, 4]])
        bad = g[[1, 3]]
        assert (bad == -1).all() if g.dtype == torch.int32 else torch.isnan(bad).all()
    d = ds.token_logprobs_backward(y, _tokens(5, 3001, 2), got[2], g_logp=torch.ones(5, device="cuda"))
    assert torch.isnan(d[[1, 3]]).all() and torch.isfinite(d[[0, 2, 4]]).all()


def test_tokens_absent_and_out_of_range():
    x = ref.logits(4, 600, torch.bfloat16, 5)
    tok = torch.tensor([-1, 600, -2, 599], dtype=torch.int32, device="cuda")
    _check(x, tok, 3)
    lp, H, lse, *_ = ds.token_logprobs(x, tok)
    g = ds.token_logprobs_backward(x, tok, lse, H, torch.ones(4, device="cuda"))
    assert (g[0] == 0).all() and torch.isnan(g[1]).all() and torch.isnan(g[2]).all() and torch.isfinite(g[3]).all()


def test_a_bad_token_of_an_empty_row_is_reported():
    x = ref.logits(4, 600, torch.float32, 5)
    x[:3] = -math.inf
    tok = torch.tensor([600, 3, -1, 4], dtype=torch.int32, device="cuda")
    lp, H, lse, *_ = ds.token_logprobs(x, tok)
    one = torch.ones(4, device="cuda")
    g = ds.token_logprobs_backward(x, tok, lse, H, one, one)
    assert torch.isnan(lp[0]) and torch.isnan(g[0]).all()
    assert (g[1:3] == 0).all() and torch.isfinite(g[3]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V", [(1, 1), (4, 33), (6, 4099), (3, 50257), (1, 262144)])
@pytest.mark.parametrize("entropy", [False, True])
def test_backward_against_64_bits(dtype, N, V, entropy):
    x = ref.logits(N, V, dtype, N + V)
    tok = _tokens(N, V, 4)
    if N > 3:
        tok[1] = -1
        x[2, ::3] = -math.inf
        tok[2] = 1
    _, H, lse, *_ = ds.token_logprobs(x, tok)
    gl = torch.randn(N, device="cuda")
    gh = torch.randn(N, device="cuda") if entropy else None
    got = ds.token_logprobs_backward(x, tok, lse, H, gl, gh)
    assert got.dtype == dtype
    want, size = ref.logprobs_backward(x, tok, lse, H, gl, gh if entropy else torch.zeros_like(gl))
    ref.assert_close(got, want, 4 * ref.U * size + 2 * ref.HALF[dtype] * want.abs() + ref.TINY[dtype], "gradient")
    inplace = x.clone()
    assert ds.token_logprobs_backward(inplace, tok, lse, H, gl, gh, out=inplace) is inplace
    assert torch.equal(inplace.nan_to_num(), got.nan_to_num())


def test_backward_against_differences():
    N, V, h = 3, 40, 1e-6
    x = ref.logits(N, V, torch.float32, 9, sigma=1.0)
    tok, gl, gh = _tokens(N, V, 4), torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    _, H, lse, *_ = ds.token_logprobs(x, tok)
    got = ds.token_logprobs_backward(x, tok, lse, H, gl, gh).double()

    def f(z):
        lp, e, *_ = ref.logprobs(z, tok, 0)
        return gl.double() * lp + gh.double() * e

    for v in range(V):
        e = torch.zeros(N, V, dtype=torch.float64, device="cuda")
        e[:, v] = h
        diff = (f(x.double() + e) - f(x.double() - e)) / (2 * h)
        # (64-bit differences: a truncation of about h^2 and a rounding of about 1e-16 * 10 / h)
        assert (diff - got[:, v]).abs().max() < 1e-5


def test_ragged_rows():
    B, R, V = 5, 4, 2003
    x = ref.logits(B * R, V, torch.float32, 1).view(B, R, V)
    tok = _tokens(B * R, V, 1).view(B, R)
    rows = torch.tensor([0, 1, 4, 9, 2], dtype=torch.int32, device="cuda")
    x[0, 0] = math.nan                    # not counted, so not read
    want = ds.token_logprobs(x, tok, top_k=6)
    got = ds.token_logprobs(x, tok, top_k=6, rows=rows)
    on = torch.arange(R, device="cuda")[None] < rows[:, None]
    for g, w, fill in zip(got, want, (0, 0, 0, -1, -math.inf)):
        assert torch.equal(g[on], w[on]) and (g[~on] == fill).all()
    d = ds.token_logprobs_backward(x, tok, got[2], got[1], torch.ones(B, R, device="cuda"),
                                   torch.ones(B, R, device="cuda"), rows=rows)
    assert (d[~on] == 0).all() and torch.isfinite(d).all() and (d[on] != 0).any(-1).all()


def test_emitted_tokens():
    B, G, V, K = 6, 5, 3011, 8
    T = ref.logits(B * (G + 1), V, torch.float32, 2).view(B, G + 1, V)
    x, tok = _tokens(B * G, V, 3).view(B, G), _tokens(B, V, 4)
    n = torch.tensor([0, 5, 2, -1, 7, 3], dtype=torch.int32, device="cuda")
    got = ds.emitted_logprobs(T, x, n, tok, top_k=K)
    j = torch.arange(G + 1, device="cuda")[None]
    held = n.clamp(max=G)
    tokens = torch.where(j < held[:, None], torch.cat([x, x[:, :1]], 1), tok[:, None]).to(torch.int32).contiguous()
    want = ds.token_logprobs(T, tokens, top_k=K, rows=(held + 1).clamp(min=0).to(torch.int32))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_emitted_tokens_of_a_round():
    from speculative_decoding_02_gb300 import workloads as wl

    w = wl.custom(B=16, gamma=4, V=4096, r=256, H=64, wdtype=torch.bfloat16, u_sigma=3.0, seed=5)
    inp = wl.make_inputs(w, 0, "cuda")
    out = ds.round(inp["U"], inp["T"], inp["W1"], inp["W2"], inp["h"], inp["w"], inp["anchor"], seed=w.seed,
                   sps=inp["sps"], mode=w.mode)
    logp, H, lse, idx, top = ds.emitted_logprobs(inp["T"], out.x, out.n, out.tok, top_k=3)
    n = out.n.tolist()
    assert any(n)
    for b in range(w.B):
        seq = out.x[b, :n[b]].tolist() + [int(out.tok[b])]
        rows = inp["T"][b, :n[b] + 1].double()
        want = torch.log_softmax(rows, -1)[torch.arange(n[b] + 1), torch.tensor(seq)]
        assert (logp[b, :n[b] + 1].double() - want).abs().max() < 2 ** -24 * (4096 / 512 + 50 + 3 * 40 + 4 * 40)
        assert (logp[b, n[b] + 1:] == 0).all() and (idx[b, n[b] + 1:] == -1).all()


def test_shapes():
    # leading dimensions of any number, among them none
    x = ref.logits(6, 777, torch.float16, 3)
    tok = _tokens(6, 777, 1)
    want = ds.token_logprobs(x, tok, top_k=4)
    got = ds.token_logprobs(x.view(3, 1, 2, 777), tok.view(3, 1, 2), top_k=4)
    assert got[0].shape == (3, 1, 2) and got[3].shape == (3, 1, 2, 4)
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    one = ds.token_logprobs(x[0], tok[0], top_k=4)
    assert one[0].shape == () and one[3].shape == (4,)
    d = ds.token_logprobs_backward(x[0], tok[0], one[2], g_logp=torch.ones((), device="cuda"))
    assert d.shape == (777,)
    # a part of a vocabulary, and requests of which a part is taken
    assert torch.equal(ds.token_logprobs(x[:, 5:], tok.clamp(max=700))[2],
                       ds.token_logprobs(x[:, 5:].contiguous(), tok.clamp(max=700))[2])


def test_no_rows():
    x = torch.empty((0, 100), device="cuda")
    tok = torch.empty((0,), dtype=torch.int32, device="cuda")
    out = ds.token_logprobs(x, tok, top_k=3)
    assert out[0].shape == (0,) and out[3].shape == (0, 3)
    assert ds.token_logprobs_backward(x, tok, out[2]).shape == (0, 100)


def test_refusals():
    x = ref.logits(4, 100, torch.float32, 1)
    tok = _tokens(4, 100, 1)
    for bad in (dict(tokens=tok[:3]), dict(tokens=tok.long()), dict(top_k=101), dict(top_k=-1),
                dict(logits=x.double()), dict(logits=x.cpu()), dict(logits=x.t()), dict(tokens=tok.cpu()),
                dict(tokens=None), dict(rows=tok), dict(logits=x[:1].expand(4, 100))):
        with pytest.raises((ValueError, TypeError)):
            ds.token_logprobs(**{"logits": x, "tokens": tok, **bad})
    with pytest.raises(ds.DSparkError) as e:
        ds.token_logprobs(ref.logits(1, 200, torch.float32, 1), tok[:1], top_k=129)
    assert e.value.code == ds.ERR_UNSUPPORTED
    with pytest.raises(ValueError):       # a gap between requests: rows are not a fixed distance apart
        ds.token_logprobs(x.view(2, 2, 100)[:, :1].expand(2, 2, 100), tok.view(2, 2))
    lse = ds.token_logprobs(x, tok)[2]
    g = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):       # overlapping, but not the same tensor
        buf = torch.empty(500, device="cuda")
        ds.token_logprobs_backward(buf[:400].view(4, 100), tok, lse, g_logp=g, out=buf[4:404].view(4, 100))
    with pytest.raises(ValueError):
        ds.token_logprobs_backward(x, tok, lse, g_entropy=g)
    with pytest.raises(TypeError):
        ds.token_logprobs_backward(x, tok, lse, g_logp=g, out=torch.empty_like(x, dtype=torch.bfloat16))


def test_sizes_past_32_bits_are_refused():
    # (their low 32 bits are a size that would be taken)
    big = torch.empty((1, 2 ** 32 + 8), dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: ds.token_logprobs(big, tok), lambda: ds.token_logprobs(big[:, :2 ** 31], tok)):
        with pytest.raises(ds.DSparkError) as e:
            call()
        assert e.value.code == ds.ERR_UNSUPPORTED
    del big
    torch.cuda.empty_cache()


def test_streams_and_graphs():
    x = [ref.logits(40, 30011, torch.bfloat16, s) for s in range(2)]
    tok = _tokens(40, 30011, 1)
    want = [ds.token_logprobs(v, tok, top_k=9) for v in x]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):                    # two streams at once
        with torch.cuda.stream(streams[i % 2]):
            got.append(ds.token_logprobs(x[i % 2], tok, top_k=9))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    static = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ds.token_logprobs(static, tok, top_k=9)
        d = ds.token_logprobs_backward(static, tok, out[2], out[1], out[0], out[1])
    for v, w in zip(x, want):
        static.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
        assert torch.equal(d, ds.token_logprobs_backward(v, tok, w[2], w[1], w[0], w[1]))
