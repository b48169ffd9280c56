"""Distillation from a teacher's top logits against plain forms in 64 bits:
loss, statistics and gradient, in one call and apart, over types, sizes,
strides, temperatures, both treatments of the teacher's tail, ragged and empty
rows, absent and repeated entries, refusals, streams and graphs."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def _teacher(S, K, tau, tail, seed, share=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    noise = torch.empty(S.shape, device="cuda").normal_(0, 1, generator=g)
    top = (S.float() + noise).nan_to_num(neginf=-1e4).topk(K)
    tl = None
    if tail:
        part = 0.3 + 0.6 * torch.rand(S.shape[0], generator=g, device="cuda") if share is None else \
            torch.full((S.shape[0],), share, device="cuda")
        tl = torch.logsumexp(top.values / tau, -1) - part.log()
    w = torch.rand(S.shape[0], generator=g, device="cuda") + 0.1
    return top.indices.to(torch.int32), top.values, tl, w


def _check(S, idx, val, tau, tl, w, gdtype=None):
    N, V = S.shape
    gd = S.dtype if gdtype is None else gdtype
    loss, stats, grad = ds.distill_loss(S, idx, val, temperature=tau, teacher_lse=tl, weight=w, grad=True,
                                        grad_dtype=gdtype)
    want = ref.distill(S, idx, val, tau, tl, w)
    fin = S.double().nan_to_num(neginf=0.0) / tau
    span = min(120.0, float((fin.amax(-1) - fin.amin(-1)).max()))
    # (1 / tau in float32, its product with log2 e and with a logit: three more steps of |z|)
    e = ref.base_error(V, span) + 4 * ref.U * (float(fin.abs().max()) + float((val / tau).abs().nan_to_num(posinf=0).max()))
    e += idx.shape[1] * ref.U
    ref.assert_close(loss, want[0], e * want[3], "loss")
    ref.assert_close(stats, want[1], e + 2 * ref.U * want[1].abs().nan_to_num(posinf=0.0), "stats")
    tol = e * want[4] + 2 * ref.HALF[gd] * want[2].abs() + ref.TINY[gd]
    ref.assert_close(grad, want[2], tol, "gradient")
    only = ds.distill_loss(S, idx, val, temperature=tau, teacher_lse=tl)
    assert only[2] is None
    # (the number of CTAs of a row, and so the order of its sums, may differ without the gradient)
    ref.assert_close(only[0], want[0], e * want[3], "loss alone")
    g = w if w is not None else torch.ones(N, device="cuda")
    back = ds.distill_loss_backward(S, idx, val, stats, g, temperature=tau, teacher_lse=tl, grad_dtype=gdtype)
    # a statistic is rounded once more: two steps of it, times tau
    e2 = e + 4 * ref.U * float(want[1].abs().nan_to_num(posinf=0.0).max())
    ref.assert_close(back, want[2], tol + e2 * want[4], "gradient alone")
    return loss, stats, grad


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N,V,K,tau", [(1, 1, 1, 1.0), (3, 5, 2, 2.0), (2, 130, 128, 0.7), (5, 4099, 64, 1.0),
                                       (4, 50257, 50, 1.5), (1, 151936, 64, 1.0), (310, 2051, 7, 4.0),
                                       (2, 300007, 16, 1.0), (1, 2097152, 100, 1.0), (160, 261000, 5, 1.0)])
def test_against_64_bits(dtype, tail, N, V, K, tau):
    S = ref.logits(N, V, dtype, N * V)
    _check(S, *(lambda i, v, t, w: (i, v, tau, t, w))(*_teacher(S, K, tau, tail, V)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N,V", [(1300, 3), (1301, 41), (1300, 1037)])
def test_more_rows_than_run_at_once(dtype, tail, N, V):
    S = ref.logits(N, V, dtype, N)
    i, v, t, w = _teacher(S, min(V, 9), 1.0, tail, V)
    _check(S, i, v, 1.0, t, w)


@pytest.mark.parametrize("tail", [False, True])
def test_bf16_gradient_of_fp32_logits(tail):
    S = ref.logits(5, 3001, torch.float32, 1)
    i, v, t, w = _teacher(S, 20, 1.0, tail, 2)
    _check(S, i, v, 1.0, t, w, torch.bfloat16)
    _check(S[:4, :3000].contiguous(), i.clamp(max=2999)[:4].contiguous(), v[:4].contiguous(), 1.0,
           None if t is None else t[:4].contiguous(), None, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("off,pad", [(1, 0), (3, 6), (0, 1)])
def test_strided_rows(dtype, tail, off, pad):
    buf = ref.logits(6, 2000 + off + pad, dtype, 3)
    S = buf[:, off:off + 2000]
    i, v, t, w = _teacher(S, 30, 1.0, tail, 2)
    keep = buf.clone()
    _check(S, i, v, 1.0, t, w)
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
def test_masked_empty_absent_and_repeated(dtype, tail):
    N, V, K = 9, 1500, 8
    S = ref.logits(N, V, dtype, 11)
    i, v, t, w = _teacher(S, K, 1.0, tail, 4)
    S[0] = -math.inf                              # nothing left in the student
    S[1, ::2] = -math.inf
    i[1] = torch.arange(1, 2 * K, 2, dtype=torch.int32, device="cuda")
    S[2] = torch.finfo(dtype).min                 # uniform
    S[3, 5:] = torch.finfo(dtype).min
    i[3] = torch.arange(K, dtype=torch.int32, device="cuda").clamp(max=4)
    i[4, 3:] = -1                                 # absent entries
    i[5] = -1                                     # no teacher: the row does not count
    i[6] = i[6, 0]                                # one index K times
    i[7, 1] = i[7, 0]
    v[8, 2] = -math.inf                           # an entry without mass
    loss, stats, grad = _check(S, i, v, 1.0, t, w)
    assert loss[0] == 0 and (grad[0] == 0).all() and loss[5] == 0 and (grad[5] == 0).all()
    # a kept entry that the student masks: infinite loss, finite gradient
    S[1, 1] = -math.inf
    loss, _, grad = ds.distill_loss(S, i, v, teacher_lse=t, grad=True)
    assert loss[1] == math.inf and torch.isfinite(grad.float()).all()


def test_whole_vocabulary_kept_and_mass_near_one():
    # K = V: nothing is left outside; and a student whose kept entries hold all
    # but 1e-6 of its mass, which 1 - sum q would lose in float32
    S = ref.logits(3, 40, torch.float32, 1)
    i = torch.stack([torch.randperm(40, device="cuda") for _ in range(3)]).to(torch.int32)
    v = torch.randn(3, 40, device="cuda")
    loss, stats, grad = ds.distill_loss(S, i, v, teacher_lse=torch.logsumexp(v.double(), -1).float() - 1e-3, grad=True)
    assert (stats[:, 1] == -math.inf).all() and torch.isfinite(loss).all() and torch.isfinite(grad).all()
    S = torch.full((2, 5000), -9.0, device="cuda")
    S[:, :4] = 14.0
    idx = torch.arange(4, dtype=torch.int32, device="cuda").expand(2, 4).contiguous()
    val = torch.zeros(2, 4, device="cuda")
    tl = torch.full((2,), math.log(4.0) + 1e-3, device="cuda")
    _check(S, idx, val, 1.0, tl, None)


def test_against_differences():
    N, V, K, h = 4, 30, 5, 1e-6
    S = ref.logits(N, V, torch.float32, 3, sigma=1.0)
    for tail in (False, True):
        i, v, t, w = _teacher(S, K, 2.0, tail, 5)
        _, _, grad = ds.distill_loss(S, i, v, temperature=2.0, teacher_lse=t, weight=w, grad=True)
        for u in range(V):
            e = torch.zeros(N, V, dtype=torch.float64, device="cuda")
            e[:, u] = h
            up, dn = (ref.distill(S.double() + s * e, i, v, 2.0, t, None)[0] for s in (1, -1))
            assert ((up - dn) / (2 * h) * w.double() - grad[:, u].double()).abs().max() < 1e-5


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
def test_in_place(dtype, tail):
    for N, V in ((3, 40961), (700, 2049), (2, 262144)):
        S = ref.logits(N, V, dtype, 3)
        i, v, t, w = _teacher(S, 24, 1.0, tail, 5)
        loss, stats, grad = ds.distill_loss(S, i, v, teacher_lse=t, weight=w, grad=True)
        a, b = S.clone(), S.clone()
        got = ds.distill_loss(a, i, v, teacher_lse=t, weight=w, grad=True, out=a)
        assert got[2] is a and torch.equal(a, grad) and torch.equal(got[0], loss) and torch.equal(got[1], stats)
        want = ds.distill_loss_backward(S, i, v, stats, w, teacher_lse=t)
        assert torch.equal(ds.distill_loss_backward(b, i, v, stats, w, teacher_lse=t, out=b), want)


def test_ragged_rows():
    B, R, V, K = 5, 4, 3003, 6
    S = ref.logits(B * R, V, torch.bfloat16, 1)
    i, v, t, w = _teacher(S, K, 1.0, True, 5)
    S = S.view(B, R, V)
    shape = lambda a: a.view(B, R, *a.shape[1:])
    i, v, t, w = map(shape, (i, v, t, w))
    rows = torch.tensor([0, 1, 4, 9, 2], dtype=torch.int32, device="cuda")
    S[0, 0] = math.nan
    full = ds.distill_loss(S, i, v, teacher_lse=t, weight=w, grad=True)
    got = ds.distill_loss(S, i, v, teacher_lse=t, weight=w, grad=True, rows=rows)
    back = ds.distill_loss_backward(S, i, v, got[1], w, teacher_lse=t, rows=rows)
    on = torch.arange(R, device="cuda")[None] < rows[:, None]
    for a, b in zip(got, full):
        assert torch.equal(a[on], b[on]) and (a[~on] == 0).all()
    assert (back[~on] == 0).all() and torch.isfinite(back.float()).all()


def test_bad_rows_are_reported():
    S = ref.logits(5, 999, torch.float32, 1)
    i, v, t, w = _teacher(S, 6, 1.0, True, 5)
    clean = ds.distill_loss(S, i, v, teacher_lse=t, grad=True)
    S[0, 998] = math.nan
    S[1, 3] = math.inf
    i[2, 1] = 999
    i[3, 5] = -2
    loss, stats, grad = ds.distill_loss(S, i, v, teacher_lse=t, grad=True)
    back = ds.distill_loss_backward(S, i, v, clean[1], torch.ones(5, device="cuda"), teacher_lse=t)
    assert torch.isnan(loss[:4]).all() and torch.isnan(grad[:4]).all()
    assert torch.isnan(back[2:4]).all() and torch.isfinite(back[4]).all()
    assert torch.equal(loss[4], clean[0][4]) and torch.equal(grad[4], clean[2][4])


@pytest.mark.parametrize("tail", [False, True])
def test_a_bad_index_in_an_empty_row_is_reported(tail):
    S = ref.logits(3, 700, torch.float32, 1)
    i, v, t, _ = _teacher(S, 6, 1.0, tail, 5)
    S[0] = S[1] = -math.inf
    i[0, 2] = 700
    loss, stats, grad = ds.distill_loss(S, i, v, teacher_lse=t, grad=True)
    back = ds.distill_loss_backward(S, i, v, stats, torch.ones(3, device="cuda"), teacher_lse=t)
    assert torch.isnan(loss[0]) and torch.isnan(grad[0]).all() and torch.isnan(back[0]).all()
    assert loss[1] == 0 and (grad[1] == 0).all() and (back[1] == 0).all()
    assert torch.isfinite(grad[2]).all() and torch.isfinite(back[2]).all()


def test_top_alternatives_are_a_teacher():
    # the target's own alternatives, kept by token_logprobs, as the teacher at
    # temperature 1: at the same logits loss and gradient vanish up to rounding
    T = ref.logits(6, 5003, torch.float32, 8)
    _, _, lse, idx, lp = ds.token_logprobs(T, torch.zeros(6, dtype=torch.int32, device="cuda"), top_k=40)
    zero = torch.zeros(6, device="cuda")
    loss, stats, grad = ds.distill_loss(T, idx, lp, teacher_lse=zero, grad=True)
    e = ref.base_error(5003, 40.0) + 64 * ref.U + 2 * ref.U * float(lse.abs().max())
    # d(p log(p / q)) is first order in the log probabilities' error, p times it, and so is each gradient
    assert loss.abs().max() < 4 * e and grad.abs().max() < 4 * e
    ref.assert_close(stats[:, 0], lse.double(), e + 2 * ref.U * lse.abs().double(), "lse")


@pytest.mark.parametrize("tau", [1e-30, 1e30])
def test_extreme_temperatures(tau):
    # hot: every entry has the same probability, to a relative 1e-29; cold: the
    # largest entry has all of it, on both sides
    N, V, K = 3, 1500, 8
    S = torch.rand((N, V), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    S[:, 7] = 2.0
    top = S.topk(K)
    i, v = top.indices.to(torch.int32), top.values
    loss, stats, grad = ds.distill_loss(S, i, v, temperature=tau, grad=True)
    back = ds.distill_loss_backward(S, i, v, stats, torch.ones(N, device="cuda"), temperature=tau)
    e = ref.base_error(V, 0.0) + K * ref.U
    if tau > 1:
        want = torch.full((N, V), 1.0 / V, dtype=torch.float64, device="cuda")
        want.scatter_add_(1, top.indices, torch.full((N, K), -1.0 / K, dtype=torch.float64, device="cuda"))
        want /= float(torch.tensor(tau))
        ref.assert_close(loss, torch.full((N,), math.log(V / K), dtype=torch.float64, device="cuda"), e * (2 + 2 * math.log(V)),
                         "loss")
        # (4 U log V more for the rounded lse)
        for g in (grad, back):
            ref.assert_close(g, want, (e + 4 * ref.U * math.log(V)) * (1.0 / V + 1.0 / K) / tau, "gradient")
    else:
        assert (loss == 0).all() and (grad == 0).all() and (back == 0).all()


def test_no_rows_and_refusals():
    S = ref.logits(4, 100, torch.float32, 1)
    i, v, t, w = _teacher(S, 6, 1.0, True, 5)
    e = ds.distill_loss(S[:0], i[:0], v[:0], grad=True)
    assert e[0].shape == (0,) and e[1].shape == (0, 2) and e[2].shape == (0, 100)
    for bad in (dict(top_idx=i[:3]), dict(top_idx=i.long()), dict(top_val=v.double()), dict(top_val=v[:, :5]),
                dict(teacher_lse=t[:3]), dict(weight=w.double()), dict(temperature=0.0), dict(temperature=math.inf),
                dict(temperature=math.nan), dict(logits=S.double()), dict(rows=i[:, 0]), dict(logits=S.cpu()),
                dict(out=S, grad=False), dict(out=S[:3], grad=True), dict(grad=True, grad_dtype=torch.int8)):
        with pytest.raises((ValueError, TypeError)):
            ds.distill_loss(**{"logits": S, "top_idx": i, "top_val": v, "teacher_lse": t, "weight": w, **bad})
    for kw in (dict(logits=S.bfloat16(), grad_dtype=torch.float32), dict(logits=S, grad_dtype=torch.float16)):
        with pytest.raises(ds.DSparkError) as err:
            ds.distill_loss(top_idx=i, top_val=v, grad=True, **kw)
        assert err.value.code == ds.ERR_UNSUPPORTED
    big = torch.zeros(1, 300, device="cuda")
    with pytest.raises(ds.DSparkError) as err:
        ds.distill_loss(big, torch.zeros(1, 129, dtype=torch.int32, device="cuda"), torch.zeros(1, 129, device="cuda"))
    assert err.value.code == ds.ERR_UNSUPPORTED


def test_streams_and_graphs():
    data = []
    for s in range(2):
        S = ref.logits(60, 20011, torch.float32, s)
        data.append((S, *_teacher(S, 12, 1.0, True, s)))
    call = lambda d: ds.distill_loss(d[0], d[1], d[2], teacher_lse=d[3], weight=d[4], grad=True)
    want = [call(d) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(call(data[k % 2]))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2]))
    static = [a.clone() for a in data[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for d, w in zip(data, want):
        for a, b in zip(static, d):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
