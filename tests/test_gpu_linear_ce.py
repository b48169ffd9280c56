"""Cross entropy of hidden states under an output head, and its gradients,
against plain forms in 64 bits: sizes, types, rows that do not count, strides,
several pieces of the vocabulary, refusals, streams and graphs."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

F64 = torch.float64
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def _inputs(B, G, V, D, dtype, seed=0, masked=0.0, ragged=False):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + V + D)
    def normal(shape, s):
        return torch.empty(shape, device="cuda").normal_(0, s, generator=g)
    W = normal((V, D), 2 / math.sqrt(D)).to(dtype)
    t = torch.randint(0, V, (B, G), generator=g, device="cuda", dtype=torch.int32)
    h = (normal((B, G, D), 1.0) + 2 * torch.rand((B, G, 1), generator=g, device="cuda") * W[t.long()].float()).to(dtype)
    t[torch.rand((B, G), generator=g, device="cuda") < masked] = -1
    rows = torch.randint(0, G + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    g_loss, g_lse = normal((B, G), 1.0), normal((B, G), 0.1)
    return h, W, t, rows, g_loss, g_lse


def _live(t, rows, V):
    on = (t >= 0) & (t < V)
    if rows is not None:
        on &= torch.arange(t.shape[1], device=t.device) < rows[:, None]
    return on


def _plain(h, W, t, rows):
    """loss, lse [B, G] in 64 bits, bounds of both, and what the gradients need."""
    V, D = W.shape
    on = _live(t, rows, V)
    x, w, tok = h[on].to(F64), W.to(F64), t[on].long()
    z = x @ w.T
    # products are exact; the tensor cores add 16 at a time, each addition off by
    # at most a step of the sum of the terms' sizes so far, the sums of chunks by half a step
    tz = 2 * ref.U * (D / 16 + 20) * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(z, -1)
    picked = z.gather(1, tok[:, None]).squeeze(1)
    # 2^x is off by 2^-22, its argument by half a step of |z|, the maximum and
    # the results by a few steps of their size; a loss has one row's fp32 dot product besides
    top = z.abs().amax(-1)
    tl = tz.amax(-1) + 2.0 ** -21 + ref.U * (8 * (lse.abs() + top) + V / 512 + 80)
    def whole(v):
        out = torch.zeros(t.shape, dtype=F64, device=t.device)
        out[on] = v
        return out
    tloss = tl + tz.gather(1, tok[:, None]).squeeze(1) + ref.U * 8 * picked.abs()
    return whole(lse - picked), whole(lse), whole(tloss), whole(tl), (on, x, w, tok, z, tz)


def _check_loss(h, W, t, rows, **kw):
    loss, lse = ds.linear_cross_entropy(h, W, t, rows=rows, **kw)
    want, wlse, tloss, tlse, parts = _plain(h, W, t, rows)
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == lse.shape == t.shape
    ref.assert_close(lse, wlse, tlse, "lse")
    ref.assert_close(loss, want, tloss, "loss")
    return loss, lse, parts


def _gradients(h, W, t, lse, g_loss, g_lse, parts):
    """dh, dW in 64 bits from the given lse, and their bounds."""
    on, x, w, tok, z, tz = parts
    half, tiny = ref.HALF[h.dtype], ref.TINY[h.dtype]
    gl = g_loss[on].to(F64)[:, None]
    up = gl if g_lse is None else gl + g_lse[on].to(F64)[:, None]
    l = lse[on].to(F64)[:, None]
    p = torch.exp(z - l)
    s = p * up
    s.scatter_add_(1, tok[:, None], -gl)
    # a slope before its rounding: the logit's error, the exponent's (a few
    # steps of |z| and of the lse), 2^-22 of 2^x; then half a step of it (of
    # fp16 at least half a step of the smallest of them, which is 2^-24 where the
    # largest |g| is about 2^14, so 2^-38 of it)
    e = p * up.abs() * (tz + ref.U * 4 * (z.abs() + l.abs()) + 2.0 ** -21) + 4 * ref.U * s.abs()
    if h.dtype == F16 and s.numel():
        e = e + 2.0 ** -38 * max(float(gl.abs().max()), float(up.abs().max()))
    r = half * s.abs()
    if on.any():
        V, N = w.shape[0], x.shape[0]
        if N <= 128:   # the remainder of the token's slope is a slope of its own, rounded in turn
            r.scatter_(1, tok[:, None], half * r.gather(1, tok[:, None]))
        er = e + r
        dW = s.T @ x
        tW = er.T @ x.abs() + 2 * ref.U * (N / 16 + 20) * (s.abs().T @ x.abs())
        dh = s @ w
        r.scatter_(1, tok[:, None], 0.0)   # (what the rounding of the token's slope took is added)
        er = e + r
        th = er @ w.abs() + 2 * ref.U * (V / 16 + 40) * (s.abs() @ w.abs())
    else:
        dW, tW = torch.zeros_like(w), torch.zeros_like(w)
        dh = th = torch.zeros((0, w.shape[1]), dtype=F64, device=w.device)
    def whole(v):
        out = torch.zeros(h.shape, dtype=F64, device=h.device)
        out[on] = v
        return out
    return whole(dh), dW, whole(th + half * dh.abs() + tiny), tW + half * dW.abs() + tiny


def _check_backward(h, W, t, rows, g_loss, g_lse, want_dh=True, want_dW=True, **kw):
    _, lse, parts = _check_loss(h, W, t, rows)
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse=g_lse, rows=rows, dh=want_dh, dW=want_dW, **kw)
    wh, ww, th, tw = _gradients(h, W, t, lse, g_loss, g_lse, parts)
    assert (dh is not None) == want_dh and (dW is not None) == want_dW
    for got, want, tol, what in ((dh, wh, th, "dh"), (dW, ww, tw, "dW")):
        if got is None:
            continue
        assert got.dtype == h.dtype and got.shape == want.shape
        ref.assert_close(got, want, tol, what)
        if float(want.norm()) > 0 and W.shape[0] > 1:
            # of the two roundings each takes at most half a step of the 2-norm.  (With one entry every
            # slope is up e^(z - lse) - g_loss with z = lse but for the fp32 steps of both, U |z| each: zero
            # without a g_lse, and want holds those steps alone, so that no bound relative to it holds; the
            # bound of each value above does.)
            assert float((got.to(F64) - want).norm() / want.norm()) < 2 * ref.HALF[h.dtype], what
    return dh, dW


SHAPES = [(1, 1, 1, 8), (1, 1, 300, 64), (3, 2, 257, 72), (16, 4, 4096, 128), (130, 2, 1000, 264), (43, 7, 5003, 136),
          (5, 3, 70001, 64), (64, 2, 900, 72), (43, 3, 900, 72), (300, 1, 129, 1032), (1, 16, 256, 2560), (257, 1, 50257, 192), (700, 5, 2056, 520)]


@pytest.mark.parametrize("B,G,V,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_loss_against_64_bits(B, G, V, D, dtype):
    h, W, t, _, _, _ = _inputs(B, G, V, D, dtype)
    _check_loss(h, W, t, None)


@pytest.mark.parametrize("B,G,V,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("what", ["both", "dh", "dW"])
def test_backward_against_64_bits(B, G, V, D, dtype, what):
    h, W, t, _, g_loss, g_lse = _inputs(B, G, V, D, dtype, 1)
    _check_backward(h, W, t, None, g_loss, g_lse if what != "dW" else None, what != "dW", what != "dh")


@pytest.mark.parametrize("masked", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("B,G,V,D", [(1, 1, 40, 16), (90, 7, 1000, 72), (600, 3, 300, 264), (1100, 3, 300, 136)])
def test_rows_that_do_not_count(B, G, V, D, masked, ragged):
    h, W, t, rows, g_loss, g_lse = _inputs(B, G, V, D, BF16, 2, masked, ragged)
    off = ~_live(t, rows, V)
    # what stands in rows that do not count has no part in anything
    h[off] = math.nan
    g_loss[off], g_lse[off] = math.nan, math.inf
    dh, dW = _check_backward(h, W, t, rows, g_loss, g_lse)
    assert (dh[off] == 0).all() and torch.isfinite(dW).all()


def test_lens_beyond_the_group_and_below_zero():
    h, W, t, _, g_loss, g_lse = _inputs(4, 5, 100, 64, BF16, 3)
    rows = torch.tensor([-3, 0, 5, 99], dtype=torch.int32, device="cuda")
    loss, lse = ds.linear_cross_entropy(h, W, t, rows=rows)
    assert (loss[:2] == 0).all() and (lse[:2] == 0).all()
    full, flse = ds.linear_cross_entropy(h, W, t)
    assert torch.equal(loss[2:], full[2:]) and torch.equal(lse[2:], flse[2:])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_pieces_of_the_vocabulary(dtype):
    # three pieces, the last of odd size
    h, W, t, _, g_loss, g_lse = _inputs(3, 2, 1100003, 16, dtype, 4)
    t[0, 0], t[1, 1], t[2, 0] = 0, 1100002, 524288
    for dh, dW in ((True, True), (True, False), (False, True)):
        _check_backward(h, W, t, None, g_loss, g_lse, dh, dW)


def test_many_rows_of_one_token():
    h, W, t, _, g_loss, _ = _inputs(64, 9, 500, 72, F16, 5)
    t.fill_(7)
    _check_backward(h, W, t, None, g_loss, None)


@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e5])
def test_upstream_gradients_of_any_size(scale):
    h, W, t, _, g_loss, g_lse = _inputs(20, 4, 3001, 136, BF16, 6)
    _check_backward(h, W, t, None, g_loss * scale, g_lse * scale)


def test_fp16_slopes_keep_small_probabilities():
    # probabilities near 2^-20 under gradients of a mean over many rows, which fp16 alone would drop
    h, W, t, _, g_loss, _ = _inputs(20, 4, 200000, 64, F16, 7)
    g = g_loss.abs() * 2.0 ** -12
    _, lse = ds.linear_cross_entropy(h, W, t)
    dh, _ = ds.linear_cross_entropy_backward(h, W, t, lse, g, dW=False)
    big, _ = ds.linear_cross_entropy_backward(h, W, t, lse, g * 2.0 ** 12, dW=False)
    fine = big.abs() > 2.0 ** -1   # (the small one's values are no subnormals there)
    assert fine.any() and torch.equal((dh.float() * 2.0 ** 12)[fine], big.float()[fine])


def test_zero_gradients_are_zeros():
    h, W, t, _, _, _ = _inputs(20, 4, 1000, 64, F16, 8)
    _, lse = ds.linear_cross_entropy(h, W, t)
    z = torch.zeros(t.shape, device="cuda")
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, z)
    assert (dh == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("D", [64, 136])
def test_strides(D):
    h, W, t, rows, g_loss, g_lse = _inputs(30, 4, 777, D, BF16, 9, 0.2, True)
    wide = torch.full((30, 4, D + 11), math.nan, dtype=BF16, device="cuda")
    for off in (0, 1, 8):   # rows of h at any alignment, rows of W on 16 bytes
        hs = wide[..., off:off + D]
        hs.copy_(h)
        head = torch.full((777, D + 24), math.nan, dtype=BF16, device="cuda")
        Ws = head[:, 8:8 + D]
        Ws.copy_(W)
        a, b = ds.linear_cross_entropy(hs, Ws, t, rows=rows), ds.linear_cross_entropy(h, W, t, rows=rows)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a = ds.linear_cross_entropy_backward(hs, Ws, t, b[1], g_loss, g_lse, rows)
        b = ds.linear_cross_entropy_backward(h, W, t, b[1], g_loss, g_lse, rows)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_tokens_out_of_range_are_reported():
    h, W, t, _, g_loss, _ = _inputs(6, 3, 500, 64, BF16, 10)
    bad = t.clone()
    bad[0, 0], bad[3, 2], bad[5, 1] = 500, -2, 2 ** 31 - 1
    off = ~_live(bad, None, 500)
    none = torch.where(off, -1, bad)
    ws = ds.linear_ce_workspace(18, 500, 64, "cuda")
    loss, lse = ds.linear_cross_entropy(h, W, bad, ws=ws)
    assert ds.read_status(ws) == ds.ERR_INVALID and ds.read_status(ws) == ds.OK
    assert torch.isnan(loss[off]).all() and (lse[off] == 0).all()
    a = ds.linear_cross_entropy(h, W, none)
    assert torch.equal(loss[~off], a[0][~off]) and torch.equal(lse[~off], a[1][~off])
    st = ds.head_status("cuda")
    ds.read_status(st)
    dh, dW = ds.linear_cross_entropy_backward(h, W, bad, lse, g_loss)
    assert ds.read_status(st) == ds.ERR_INVALID
    wh, ww = ds.linear_cross_entropy_backward(h, W, none, lse, g_loss)
    assert ds.read_status(st) == ds.OK
    assert torch.equal(dW, ww) and torch.equal(dh[~off], wh[~off]) and torch.isnan(dh[off]).all()


def test_values_that_are_not_finite():
    h, W, t, _, g_loss, _ = _inputs(5, 2, 300, 64, BF16, 11)
    h[1, 0, 3] = math.nan
    h[3, 1, 0] = math.inf
    loss, lse = ds.linear_cross_entropy(h, W, t)
    bad = torch.zeros((5, 2), dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[3, 1] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all()
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, dW=False)
    assert torch.isnan(dh[bad]).all() and torch.isfinite(dh[~bad]).all()


def test_a_sure_row_keeps_its_small_loss():
    # the token has all but e^-9 of the mass or so: a loss far below the lse's own step is not a difference of two large ones
    V, D = 300, 64
    W = torch.zeros((V, D), dtype=BF16, device="cuda")
    W[7, 0] = 1.0
    h = torch.zeros((4, D), dtype=BF16, device="cuda")
    h[:, 0] = torch.tensor([16.0, 18.0, 20.0, 24.0], device="cuda")
    t = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    loss, _ = ds.linear_cross_entropy(h, W, t)
    want = torch.log1p((V - 1) * torch.exp(-h[:, 0].double()))
    # the sum of exponentials, 1 + want, is held to half a step of 1 a few times over
    ref.assert_close(loss, want, 16 * ref.U, "loss")


def test_differences():
    # the gradients along a direction against differences of the 64-bit loss
    h, W, t, rows, g_loss, g_lse = _inputs(12, 5, 400, 72, BF16, 12, 0.2, True)
    dh, dW = _check_backward(h, W, t, rows, g_loss, g_lse)
    _, lse = ds.linear_cross_entropy(h, W, t, rows=rows)
    parts = _plain(h, W, t, rows)[4]
    _, _, th, tw = _gradients(h, W, t, lse, g_loss, g_lse, parts)
    g = torch.Generator(device="cuda").manual_seed(5)
    on = _live(t, rows, 400)

    def total(a, b):
        z = torch.einsum("bgd,vd->bgv", a, b)
        l = torch.logsumexp(z, -1)
        loss = l - z.gather(2, t.long().clamp(min=0)[..., None]).squeeze(-1)
        return ((g_loss.double() * loss + g_lse.double() * l) * on).sum()

    for grad, tol, which in ((dh, th, 0), (dW, tw, 1)):
        u = torch.randn(grad.shape, generator=g, device="cuda", dtype=F64)
        x = [h.double(), W.double()]
        step = 1e-4
        lo, hi = list(x), list(x)
        lo[which], hi[which] = x[which] - step * u, x[which] + step * u
        slope = (total(*hi) - total(*lo)) / (2 * step)
        # third derivatives of a log-sum-exp are at most those of its exponents' cube; the lse given is fp32
        bound = (tol * u.abs()).sum() + 1e-5 * (1 + slope.abs())
        assert abs(float((grad.double() * u).sum() - slope)) < float(bound)


def test_offsets_past_32_bits():
    V, D = 140001, 16384   # the head has 2.3e9 values
    g = torch.Generator(device="cuda").manual_seed(17)
    W = torch.empty((V, D), dtype=BF16, device="cuda").normal_(0, 2 / math.sqrt(D), generator=g)
    t = torch.tensor([[V - 1, 7, 139264]], dtype=torch.int32, device="cuda")
    h = torch.empty((1, 3, D), device="cuda").normal_(0, 1, generator=g).to(BF16)
    loss, lse = ds.linear_cross_entropy(h, W, t)
    weight = torch.ones((1, 3), device="cuda")
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, weight)
    x, parts = h[0].to(F64), W.split(8192)
    z = torch.cat([x @ w.to(F64).T for w in parts], 1)
    size = torch.cat([x.abs() @ w.to(F64).abs().T for w in parts], 1)
    want = torch.logsumexp(z, -1)
    tz = 2 * ref.U * (D / 16 + 20) * size.amax()
    ref.assert_close(lse[0], want, tz + 2.0 ** -18, "lse")
    ref.assert_close(loss[0], want - z.gather(1, t[0].long()[:, None]).squeeze(1), 2 * tz + 2.0 ** -18, "loss")
    s = torch.softmax(z, -1)
    s[torch.arange(3), t[0].long()] -= 1.0
    want = torch.zeros((3, D), dtype=F64, device="cuda")
    for k, w in enumerate(parts):
        want += s[:, 8192 * k:8192 * k + w.shape[0]] @ w.to(F64)
    assert float((dh[0].to(F64) - want).norm() / want.norm()) < 2 * ref.HALF[BF16]
    for first in (0, 131072, V - 700):   # pieces below, across and past 2^31 values
        rows = slice(first, first + 700)
        want = s[:, rows].T @ x
        assert float((dW[rows].to(F64) - want).norm() / want.norm()) < 2 * ref.HALF[BF16]


def test_results_are_reproducible():
    h, W, t, rows, g_loss, g_lse = _inputs(300, 4, 5000, 264, BF16, 13, 0.3, True)
    call = lambda: (*ds.linear_cross_entropy(h, W, t, rows=rows),
                    *ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse, rows))
    _, lse = ds.linear_cross_entropy(h, W, t, rows=rows)
    first = call()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


def test_a_dirty_workspace_of_exact_size():
    h, W, t, rows, g_loss, g_lse = _inputs(70, 4, 3000, 136, F16, 14, 0.3, True)
    want = ds.linear_cross_entropy(h, W, t, rows=rows)
    grads = ds.linear_cross_entropy_backward(h, W, t, want[1], g_loss, g_lse, rows)
    for byte in (0x00, 0x7f, 0xff):
        ws = ds.linear_ce_workspace(280, 3000, 136, "cuda")
        ws.fill_(byte)
        ws[:256].zero_()
        assert all(torch.equal(a, b) for a, b in zip(want, ds.linear_cross_entropy(h, W, t, rows=rows, ws=ws)))
        assert ds.read_status(ws) == ds.OK
        for dh, dW in ((True, True), (True, False), (False, True)):
            ws = ds.linear_ce_workspace(280, 3000, 136, "cuda", dh=dh, dW=dW)
            ws.fill_(byte)
            ws[:256].zero_()
            got = ds.linear_cross_entropy_backward(h, W, t, want[1], g_loss, g_lse, rows, dh=dh, dW=dW, ws=ws)
            assert ds.read_status(ws) == ds.OK
            if dW:
                assert torch.equal(got[1], grads[1])
            if dh and dW:
                assert torch.equal(got[0], grads[0])


def test_no_rows():
    _, W, _, _, _, _ = _inputs(1, 1, 300, 64, BF16)
    h = torch.empty((0, 3, 64), dtype=BF16, device="cuda")
    t = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    z = torch.empty((0, 3), device="cuda")
    loss, lse = ds.linear_cross_entropy(h, W, t)
    assert loss.shape == lse.shape == (0, 3)
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, z, z)
    assert dh.shape == h.shape and (dW == 0).all()


def test_one_dimension_and_none():
    h, W, t, _, g_loss, _ = _inputs(1, 6, 300, 64, BF16, 15)
    a = ds.linear_cross_entropy(h, W, t)
    b = ds.linear_cross_entropy(h[0], W, t[0])
    c = ds.linear_cross_entropy(h[0, 2], W, t[0, 2])
    assert torch.equal(a[0][0], b[0]) and c[0].shape == () and torch.equal(c[0], b[0][2])


def test_refusals():
    h, W, t, rows, g, _ = _inputs(4, 3, 300, 64, BF16, 16)
    lse = torch.zeros((4, 3), device="cuda")
    for a in ((h.float(), W, t), (h, W.half(), t), (h, W, t.long()), (h.cpu(), W, t), (h, W.cpu(), t), (h, W, t.cpu())):
        with pytest.raises((TypeError, ValueError)):
            ds.linear_cross_entropy(*a)
    for a in ((h, W[:, :56], t), (h, W, t[:, :2]), (h, W.T, t), (h.transpose(1, 2), W, t), (h, W[None], t), (h, W[:0], t)):
        with pytest.raises(ValueError):
            ds.linear_cross_entropy(*a)
    with pytest.raises(ds.DSparkError) as e:
        ds.linear_cross_entropy(h.float(), W.float(), t)
    assert e.value.code == ds.ERR_UNSUPPORTED
    with pytest.raises(ds.DSparkError) as e:
        ds.linear_cross_entropy(h[..., :60], W[:, :60], t)
    assert e.value.code == ds.ERR_UNSUPPORTED
    with pytest.raises(ds.DSparkError) as e:   # a head whose rows do not start on 16 bytes
        ds.linear_cross_entropy(h[..., :56], W[:, 4:60], t)
    assert e.value.code == ds.ERR_INVALID
    with pytest.raises(ds.DSparkError) as e:
        ds.linear_cross_entropy(h, W, t, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == ds.ERR_WORKSPACE
    with pytest.raises(ValueError):
        ds.linear_cross_entropy_backward(h, W, t, lse, g, dh=False, dW=False)
    with pytest.raises(ValueError):
        ds.linear_cross_entropy_backward(h, W, t, lse[:, :2], g)
    with pytest.raises(ValueError):
        ds.linear_cross_entropy_backward(h, W, t, lse, None)


def test_streams_and_graphs():
    data = [_inputs(40, 4, 3001, 136, BF16, s, 0.2, True) for s in range(2)]

    def call(d):
        h, W, t, rows, g_loss, g_lse = d
        loss, lse = ds.linear_cross_entropy(h, W, t, rows=rows)
        return (loss, lse, *ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse, rows))

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


@pytest.mark.parametrize("N,V,D,dtype", [(520, 50000, 64, BF16), (520, 50000, 512, BF16), (600, 50257, 136, F16), (1300, 33000, 256, BF16)])
def test_tiles_without_rows_between_tiles_with_rows(N, V, D, dtype):
    # a last row tile whose rows past N leave warps idle, and units that take the row tiles of several
    # columns in turn, each in one accumulator
    h, W, t, _, _, _ = _inputs(N, 1, V, D, dtype, 18)
    loss, lse, _ = _check_loss(h, W, t, None)
    for _ in range(40):
        again = ds.linear_cross_entropy(h, W, t)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


def test_many_rows_of_which_few_count():
    # more rows than one kernel both counts and gathers, a hundred of them live
    h, W, t, _, g_loss, g_lse = _inputs(3000, 1, 900, 136, BF16, 23)
    keep = torch.zeros_like(t, dtype=torch.bool)
    keep[torch.randperm(3000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")[:100]] = True
    t[~keep] = -1
    for dh, dW in ((True, True), (False, True), (True, False)):
        _check_backward(h, W, t, None, g_loss, g_lse, dh, dW)


@pytest.mark.parametrize("N,V,D,dtype", [(2048, 3001, 2560, BF16), (1500, 2000, 4096, F16), (5000, 60001, 1032, BF16)])
def test_dh_alone_of_more_tiles_than_pairs(N, V, D, dtype):
    # some tiles of dh whole, the others in parts (77 to 100 for 76 pairs); the last case in several pieces of the vocabulary
    h, W, t, rows, g_loss, g_lse = _inputs(N, 1, V, D, dtype, 24, 0.02)
    _check_backward(h, W, t, rows, g_loss, g_lse, True, False)


def test_a_dirty_workspace_of_dh_alone():
    h, W, t, rows, g_loss, g_lse = _inputs(128, 16, 3001, 2568, BF16, 25)
    _, lse = ds.linear_cross_entropy(h, W, t)
    want, _ = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse, dW=False)
    for byte in (0x00, 0x7f, 0xff):
        ws = ds.linear_ce_workspace(2048, 3001, 2568, "cuda", dh=True)
        ws.fill_(byte)
        ws[:256].zero_()
        got, _ = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse, dW=False, ws=ws)
        assert torch.equal(got, want) and ds.read_status(ws) == ds.OK


@pytest.mark.parametrize("N", [1, 20, 45, 130, 2100])
def test_an_infinite_entry_of_the_head_leaves_other_rows_of_dW(N):
    # every row's logit at v is -inf: probability 0, so dW[v] is 0 (and dh, 0 times -inf, NaN there)
    h, W, t, _, g_loss, g_lse = _inputs(N, 1, 700, 72, BF16, 19)
    v = 333
    t[t == v] = 1
    h[..., 5] = h[..., 5].abs() + 0.5
    W[v, 5] = -math.inf
    loss, lse = ds.linear_cross_entropy(h, W, t)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse)
    assert (dW[v] == 0).all() and torch.isfinite(dW).all()
    assert torch.isnan(dh[..., 5]).all()
    dh[..., 5] = 0
    assert torch.isfinite(dh).all()
    _, alone = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss, g_lse, dh=False)
    assert torch.equal(alone, dW)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("g", [1.0, 1.00390625, -0.7])
def test_the_remainder_of_a_slope_adds_no_infinity(dtype, g):
    # one row whose token's own entry of the head is -inf: the loss is inf, its slope there is -g exactly
    # (1.00390625 = 1 + 2^-8 leaves a remainder in bf16), and dh -g times -inf
    h, W, t, _, _, _ = _inputs(1, 1, 300, 64, dtype, 20)
    h[..., 5] = 1.0
    W[t.long().flatten(), 5] = -math.inf
    loss, lse = ds.linear_cross_entropy(h, W, t)
    assert (loss == math.inf).all() and torch.isfinite(lse).all()
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, torch.full((1, 1), g, device="cuda"))
    assert (dh[..., 5] == math.copysign(math.inf, g)).all()
    dh[..., 5] = 0
    assert torch.isfinite(dh).all() and torch.isfinite(dW).all()


def test_fp16_rows_of_very_different_upstream_gradients():
    # dh alone: a row's slopes keep their digits whatever the other rows' gradients are
    h, W, t, _, g_loss, _ = _inputs(20, 4, 3001, 64, F16, 21)
    W, g = W * 0.1, g_loss.abs() + 0.5
    g[::2] *= 2.0 ** 13
    g[1::2] *= 2.0 ** -9
    _, lse = ds.linear_cross_entropy(h, W, t)
    dh, _ = ds.linear_cross_entropy_backward(h, W, t, lse, g, dW=False)
    for b in range(20):
        parts = _plain(h[b:b + 1], W, t[b:b + 1], None)[4]
        want, _, tol, _ = _gradients(h[b:b + 1], W, t[b:b + 1], lse[b:b + 1], g[b:b + 1], None, parts)
        ref.assert_close(dh[b:b + 1], want, tol, "dh")


def test_a_logit_of_plus_infinity():
    # reported as NaN, as for rows of logits; other rows keep their loss
    h, W, t, _, g_loss, _ = _inputs(6, 2, 300, 64, BF16, 26)
    h[..., 5] = -1.0
    want = ds.linear_cross_entropy(h, W, t)
    h[2, 1, 5] = 1.0
    t[t == 17] = 18
    W[17, 5] = math.inf   # the logit of 17 is +inf in row (2, 1), -inf in the others
    bad = torch.zeros((6, 2), dtype=torch.bool, device="cuda")
    bad[2, 1] = True
    loss, lse = ds.linear_cross_entropy(h, W, t)
    assert torch.isnan(loss[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(loss[~bad]).all() and (lse[~bad] <= want[1][~bad]).all()
    dh, dW = ds.linear_cross_entropy_backward(h, W, t, lse, g_loss)
    assert torch.isnan(dh[bad]).all() and torch.isnan(dW).all()
