"""Newton-Schulz orthogonalisation against its definition in 64 bits: one step
value by value, several in the 2-norm; sizes, types, strides, edge values, streams
and graphs; and a training step whose gradients it takes."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

F64 = torch.float64
MUON = (3.4445, -4.7750, 2.0315)
H = 2.0 ** -11          # half a step of fp16, relative
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def _update(m, n, dtype=torch.float32, seed=0, kind="noise"):
    g = torch.Generator(device="cuda").manual_seed(7919 * seed + 31 * m + n)
    x = torch.randn((m, n), generator=g, device="cuda")
    if kind == "low rank":
        k = min(8, m, n)
        x = torch.randn((m, k), generator=g, device="cuda") @ torch.randn((k, n), generator=g, device="cuda") + 0.03 * x
    if kind == "rows":   # rows of sizes far apart
        x *= torch.exp(2 * torch.randn((m, 1), generator=g, device="cuda"))
    return (1e-2 * x).to(dtype)


def _fp16(x, halves):
    """The operand that a product takes: fp16 of 2^10 x, with halves the rest too."""
    h = (x * 1024).to(torch.float16).to(F64) / 1024
    return h + _fp16(x - h, False) if halves else h


def _steps(M, steps, coefficients, eps, rounded):
    a, b, c = coefficients
    X = M.to(F64)
    X = X / (X.norm() + eps)
    tall = M.shape[0] > M.shape[1]
    if tall:
        X = X.T
    halves = min(M.shape) <= 512
    for _ in range(steps):
        x = _fp16(X, halves) if rounded else X
        A = x @ x.T
        A = _fp16(A, halves) if rounded else A
        B = b * A + c * (A @ A)
        X = a * X + (_fp16(B, halves) if rounded else B) @ x
    return X.T if tall else X


def _one_step_bound(M, coefficients, eps):
    """Bound of each value after one step: every operand is off by H of itself
    (and by 2^-35, half of fp16's smallest step over 2^10), products are exact,
    sums of K terms off by a step (2 U) of the terms' sizes for each 16 of K and a
    few more; X from its halves by 2^-22 of itself; the result's own rounding."""
    a, b, c = map(abs, coefficients)
    tall = M.shape[0] > M.shape[1]
    X = M.to(F64)
    X = X / (X.norm() + eps)
    X = (X.T if tall else X)
    s, n = X.shape
    x = X.abs()
    tiny = 2.0 ** -35
    dx = H * x + tiny
    sums = lambda K: 2 * ref.U * (K / 16 + 20)
    A = X @ X.T
    absA = x @ x.T
    dA = dx @ x.T + x @ dx.T + dx @ dx.T + sums(n) * absA
    dA = dA + H * (A.abs() + dA) + tiny
    AA = A.abs() + dA
    dB = b * dA + c * (dA @ AA + A.abs() @ dA + sums(s) * (AA @ AA)) + 4 * ref.U * (b * AA + c * (AA @ AA))
    B = coefficients[1] * A + coefficients[2] * (A @ A)
    dB = dB + H * (B.abs() + dB) + tiny
    BB = B.abs() + dB
    Y = coefficients[0] * X + B @ X
    dY = dB @ (x + dx) + B.abs() @ dx + sums(s) * (BB @ (x + dx)) + a * (2.0 ** -20 * x + tiny) + 8 * ref.U * Y.abs()
    dY = dY + ref.HALF[torch.bfloat16] * (Y.abs() + dY)
    return (Y.T, dY.T) if tall else (Y, dY)


SHAPES = [(1, 1), (1, 40), (40, 1), (2, 3), (16, 16), (64, 300), (300, 64), (128, 128), (129, 257), (257, 129), (256, 512),
          (100, 5000), (5000, 100), (513, 513), (777, 1000), (1000, 777), (1280, 1536), (20011, 256), (256, 20011),
          (30000, 72), (33000, 200), (300, 17001), (20000, 500)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_one_step(m, n, dtype):
    M = _update(m, n, dtype)
    got = ds.newton_schulz(M, steps=1)
    assert got.dtype == torch.bfloat16 and got.shape == M.shape and got.is_contiguous()
    want, tol = _one_step_bound(M, MUON, 1e-7)
    ref.assert_close(got, want, tol, "one step")


@pytest.mark.parametrize("m,n", SHAPES + [(2048, 2048), (700, 151936), (151936, 256), (4096, 1100)])
@pytest.mark.parametrize("kind", ["noise", "low rank", "rows"])
def test_five_steps(m, n, kind):
    M = _update(m, n, torch.float32, 1, kind)
    got = ds.newton_schulz(M).to(F64)
    want = _steps(M, 5, MUON, 1e-7, False)
    # the products' operands rounded as they are, in 64 bits: what is left are the
    # fp32 sums (2^-24 of a term or so, up to 3.5^5 = 500 times as much after
    # the steps) and operands that round to the other neighbour for them
    same = _steps(M, 5, MUON, 1e-7, True)
    off = float((same - want).norm())
    bound = ref.HALF[torch.bfloat16] * float(want.norm()) + 1.5 * off + 2.0 ** -12 * float(want.norm())
    assert float((got - want).norm()) <= bound
    # and that is near the rounding of the result alone
    assert float((got - want).norm()) <= 2.0 ** -8 * float(want.norm())


def test_singular_values():
    M = _update(300, 500, torch.float32, 2)
    s = torch.linalg.svdvals(ds.newton_schulz(M).float())
    x = torch.linalg.svdvals(M.double() / M.double().norm())
    for _ in range(5):
        x = MUON[0] * x + MUON[1] * x ** 3 + MUON[2] * x ** 5
    # each is off by at most the 2-norm of the difference: 2^-8 of the matrix' Frobenius norm, and that is far from all of them
    assert float((torch.sort(s.double()).values - torch.sort(x).values).abs().max()) < 2.0 ** -8 * float(x.norm())


@pytest.mark.parametrize("steps,coefficients", [(1, (1.5, -0.5, 0.0)), (12, (1.5, -0.5, 0.0)), (3, (1.875, -1.25, 0.375)),
                                                (10, MUON), (7, (2.0, -1.5, 0.5))])
@pytest.mark.parametrize("m,n", [(96, 200), (400, 136), (90001, 64), (400, 20000), (600, 530)])
def test_other_coefficients(steps, coefficients, m, n):
    M = _update(m, n, torch.float32, 3)
    got = ds.newton_schulz(M, steps=steps, coefficients=coefficients).to(F64)
    want, same = (_steps(M, steps, coefficients, 1e-7, r) for r in (False, True))
    bound = (ref.HALF[torch.bfloat16] + 2.0 ** -12) * float(want.norm()) + 1.5 * float((same - want).norm())
    assert float((got - want).norm()) <= bound


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-12, 1.0, 1e12, 1e35])
def test_updates_of_any_size(scale):
    M = _update(70, 90, torch.float32, 4) * 10 * scale
    if scale == 1e-42:   # subnormal values, few of them zero: their own values count
        assert float((M != 0).float().mean()) > 0.9
    got = ds.newton_schulz(M, steps=1, eps=0.0)
    want, tol = _one_step_bound(M, MUON, 0.0)
    ref.assert_close(got, want, tol, "one step")


def test_eps():
    M = _update(20, 30, torch.float32, 5)
    for eps in (0.0, 1e-3, 1.0, 100.0):
        want, tol = _one_step_bound(M, MUON, eps)
        ref.assert_close(ds.newton_schulz(M, steps=1, eps=eps), want, tol, "eps")


def test_zeros_and_values_that_are_not_finite():
    M = torch.zeros((50, 70), device="cuda")
    assert (ds.newton_schulz(M) == 0).all()
    assert torch.isnan(ds.newton_schulz(M, eps=0.0)).all()
    M = _update(50, 70)
    M[3, 4] = math.nan
    assert torch.isnan(ds.newton_schulz(M)).all()
    M[3, 4] = math.inf   # an infinite norm: zeros, and inf / inf where it stood
    assert torch.isnan(ds.newton_schulz(M)).any()
    one = torch.zeros((50, 70), device="cuda")
    one[7, 9] = -3.0     # one singular value: the others stay zero
    got = ds.newton_schulz(one)
    x = 1.0
    for _ in range(5):
        x = MUON[0] * x + MUON[1] * x ** 3 + MUON[2] * x ** 5
    assert float(got[7, 9]) == pytest.approx(-x, rel=2.0 ** -7)
    got[7, 9] = 0
    assert (got == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(60, 77), (200, 136)])
def test_strides(dtype, m, n):
    M = _update(m, n, dtype, 6)
    want = ds.newton_schulz(M)
    for off, pad in ((0, 3), (1, 4), (4, 8)):
        wide = torch.full((m, n + off + pad), math.nan, dtype=dtype, device="cuda")
        view = wide[:, off:off + n]
        view.copy_(M)
        assert torch.equal(ds.newton_schulz(view), want)


@pytest.mark.parametrize("m,n", [(300, 260), (40000, 136), (1500, 1100)])
def test_reproducible_and_a_dirty_workspace(m, n):
    M = _update(m, n, torch.float32, 7)
    want = ds.newton_schulz(M)
    for byte in (0x00, 0x7f, 0xff):
        ws = ds.newton_schulz_workspace(m, n, "cuda")
        ws.fill_(byte)
        ws[:256].zero_()
        assert torch.equal(ds.newton_schulz(M, ws=ws), want)
        assert ds.read_status(ws) == ds.OK


@pytest.mark.parametrize("n,r", [(1040, 1024), (250, 1024)])
def test_offsets_past_32_bits(n, r):
    # r copies of a block below one another have the block's singular values times
    # sqrt(r), so the result is the block's result over sqrt(r), r times
    B = _update(2048, n, torch.bfloat16, 10)
    got = ds.newton_schulz(B.repeat(r, 1))   # 2.2e9 values (n = 1040)
    same = got.view(r, 2048, n)
    assert all(torch.equal(same[k], same[0]) for k in range(1, r, 89)) and torch.equal(same[-1], same[0])
    want = _steps(B, 5, MUON, 0.0, False) / math.sqrt(r)
    assert float((got[:2048].to(F64) - want).norm()) <= 2.0 ** -8 * float(want.norm())


def test_refusals():
    M = _update(20, 30)
    for bad in (M.double(), M.int()):
        with pytest.raises(TypeError):
            ds.newton_schulz(bad)
    for bad in (M.cpu(), M[None], M[0], M.T, M[:, ::2], M.expand(4, 20, 30)[:, 0], M[:1].expand(20, 30), None):
        with pytest.raises(ValueError):
            ds.newton_schulz(bad)
    for kw in (dict(coefficients=(1.0, math.nan, 0.0)), dict(eps=-1.0), dict(eps=math.inf), dict(coefficients=(1.0, 2.0))):
        with pytest.raises(ValueError):
            ds.newton_schulz(M, **kw)
    for kw, code in ((dict(steps=0), ds.ERR_INVALID), (dict(steps=65), ds.ERR_UNSUPPORTED),
                     (dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")), ds.ERR_WORKSPACE)):
        with pytest.raises(ds.DSparkError) as e:
            ds.newton_schulz(M, **kw)
        assert e.value.code == code
    assert ds.newton_schulz(M[:0]).shape == (0, 30) and ds.newton_schulz(M[:, :0]).shape == (20, 0)


def test_streams_and_graphs():
    data = [_update(300, 400, torch.bfloat16, s) for s in (8, 9)]
    want = [ds.newton_schulz(d) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(ds.newton_schulz(data[k % 2]))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert torch.equal(g, want[k % 2])
    static = data[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ds.newton_schulz(static)
    for d, w in zip(data, want):
        static.copy_(d)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_calls_at_once():
    # launches whose CTAs wait for one another beside others that fill the GPU, from
    # three threads on streams of their own
    import threading
    data = [_update(m, n, torch.float32, 11) for m, n in ((256, 256), (777, 1000), (4000, 64))]
    g = torch.Generator(device="cuda").manual_seed(12)
    W = torch.randn((30000, 512), device="cuda", generator=g).mul_(0.1).bfloat16()
    h = torch.randn((2048, 512), device="cuda", generator=g).bfloat16()
    t = torch.randint(0, 30000, (2048,), device="cuda", generator=g, dtype=torch.int32)
    calls = [lambda k=k: (ds.newton_schulz(data[k % 3]),) for k in range(3)] + [lambda: ds.linear_cross_entropy(h, W, t)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(first):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(24):
                k = (first + i) % 4
                if not all(torch.equal(a, b) for a, b in zip(calls[k](), want[k])):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [x.start() for x in threads]
    [x.join() for x in threads]
    assert not wrong and ds.read_status(ds.head_status("cuda")) == ds.OK


def test_a_training_step_of_draft_and_head():
    """The operators together, as a step uses them: the loss of a projection's
    hidden states under a head with the Markov head's rows beside it, the gradients,
    the update of both weights; each against its 64-bit form on the same inputs."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, G, V, D, R = 24, 5, 3001, 192, 256
    normal = lambda shape, s: torch.empty(shape, device="cuda").normal_(0, s, generator=g)
    P = normal((D, D), D ** -0.5)                               # the draft's weight
    head = normal((V, D + R), 0.1).bfloat16()                   # [W | W2]: logits h W^T + W1[prev] W2^T
    W1 = normal((V, R), 0.3).bfloat16()
    x = normal((B, G, D), 1.0).bfloat16()
    t = torch.randint(0, V, (B, G), generator=g, device="cuda", dtype=torch.int32)
    anchor = torch.randint(0, V, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    prev = torch.cat([anchor, t[:, :-1]], 1).long()
    rows = torch.randint(1, G + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    momentum = torch.zeros_like(P)

    def step(P, momentum):
        h = torch.cat([x @ P.bfloat16().T, W1[prev]], -1)
        loss, lse = ds.linear_cross_entropy(h, head, t, rows=rows)
        weight = (1.0 / rows.sum()).expand(B, G).contiguous()
        dh, dhead = ds.linear_cross_entropy_backward(h, head, t, lse, weight, rows=rows)
        dP = dh[..., :D].reshape(-1, D).float().T @ x.reshape(-1, D).float()
        momentum.mul_(0.95).add_(dP)
        return h, loss, lse, weight, dh, dhead, momentum.clone(), ds.newton_schulz(momentum)

    h, loss, lse, weight, dh, dhead, M, O = step(P, momentum)
    on = torch.arange(G, device="cuda") < rows[:, None]
    z = (h.double() @ head.double().T)
    want = torch.logsumexp(z, -1) - z.gather(2, t.long()[..., None]).squeeze(-1)
    # D + R products in fp32, as bounded for the loss alone
    size = (h.double().abs() @ head.double().abs().T).amax(-1)
    assert ((loss.double() - want).abs()[on] <= (4 * ref.U * ((D + R) / 16 + 20) * size + 2.0 ** -19)[on]).all()
    assert (loss[~on] == 0).all()
    s = torch.softmax(z, -1)
    s.scatter_add_(2, t.long()[..., None], torch.full_like(s[..., :1], -1))
    s = (s * (weight.double() * on)[..., None]).reshape(-1, V)
    for got, w in ((dh.reshape(-1, D + R), s @ head.double()), (dhead, s.T @ h.double().reshape(-1, D + R))):
        assert float((got.double() - w).norm() / w.norm()) < 2 * ref.HALF[torch.bfloat16]
    w = _steps(M, 5, MUON, 1e-7, False)
    assert float((O.double() - w).norm() / w.norm()) < 2.0 ** -8
    # the same step captured and replayed, with the update applied, and run beside it
    static_P, static_M = P.clone(), torch.zeros_like(P)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static_P, static_M)
        static_P.add_(out[-1], alpha=-0.02)
    eager_P, eager_M = P.clone(), torch.zeros_like(P)
    static_P.copy_(P)
    static_M.zero_()
    for _ in range(2):
        graph.replay()
        eager = step(eager_P, eager_M)
        eager_P.add_(eager[-1], alpha=-0.02)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)) and torch.equal(static_P, eager_P)
