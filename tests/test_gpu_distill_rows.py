"""Distillation with each row held to bounds of its own: rows whose entries
outside the kept ones are masked by finite values, rows far from zero, masked,
absent and repeated entries, and teachers that kept almost all of their mass.

The reference subtracts a row's maximum before anything else, so that log V is
not lost beside a mask of the type's lowest value, and every bound follows from
differences to that maximum, never from the size of the logits."""
import math

import pytest
import torch

import speculative_decoding_02_gb300 as ds

import _rows as ref

pytestmark = pytest.mark.gpu

F64, U = torch.float64, ref.U
FLT_MAX = torch.finfo(torch.float32).max
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_02_gb300 import build
    build.build()
    ds.library()


def f32(v):
    """A temperature as the library gets it."""
    return float(torch.tensor(v, dtype=torch.float32))


def _finite(t):
    return torch.where(torch.isfinite(t), t, torch.zeros_like(t))


def _states(z, tau):
    """Maximum, distances (z - max) / tau, log of the sum and the relative error of
    the sum for each row: base_error without its span, and five steps of a
    term's distance (x - m, 1 / tau, log2 e and two products) weighted as in the sum."""
    m = z.amax(-1, keepdim=True)
    none = m == -math.inf
    d = torch.where(none, torch.full_like(z, -math.inf), (z - torch.where(none, torch.zeros_like(m), m)) / tau)
    e = torch.exp(d)
    s = e.sum(-1, keepdim=True)
    ls = torch.where(none, torch.zeros_like(s), s.log())
    weighted = (e * _finite(d).abs()).sum(-1, keepdim=True) / s.clamp(min=1.0)
    return m, d, ls, ref.base_error(z.shape[-1], 0.0) + 5 * U * weighted


def _want(S, idx, val, tau, tlse, w):
    """(loss, its bound), (stats, their bound), (gradient, its bound, the additional
    bound of the gradient from rounded stats); tau as the library gets it."""
    N, V = S.shape
    K = idx.shape[1]
    z = S.to(F64)
    present = (idx >= 0)
    ii = idx.long().clamp(min=0)
    t = torch.where(present, val.to(F64) / tau, torch.full((N, K), -math.inf, dtype=F64, device=S.device))
    any_ = (t > -math.inf).any(-1)
    tm = torch.where(any_[:, None], t.amax(-1, keepdim=True), torch.zeros(N, 1, dtype=F64, device=S.device))
    norm = tlse.to(F64)[:, None] if tlse is not None else tm + torch.where(
        any_[:, None], torch.exp(t - tm).sum(-1, keepdim=True), torch.ones_like(tm)).log()
    lp = t - norm
    p = torch.exp(lp)
    # relative error of p_k: its argument (product, difference, rounded), the
    # kept entries' sum where it divides by one, the exponential
    ep = U * (4 * _finite(t - tm).abs() + 2 * _finite(lp).abs() + 40)
    m, d, ls, ea = _states(z, tau)
    on = any_ & (m.squeeze(1) > -math.inf)
    q = torch.exp(d - ls)
    dk = d.gather(1, ii)
    gap = torch.where(p > 0, lp - (dk - ls), torch.zeros_like(p))
    loss = (p * gap).sum(-1)
    part = p * (ea + 6 * U * (_finite(dk).abs() + ls + _finite(lp).abs()) + ep * (1 + gap.abs()) + 16 * U * gap.abs())
    eloss = torch.where(torch.isfinite(part), part, torch.zeros_like(part)).sum(-1)
    mass = torch.zeros_like(z).scatter_add_(1, ii, p * present)
    emass = torch.zeros_like(z).scatter_add_(1, ii, p * ep * present)
    inside = torch.zeros_like(z).scatter_add_(1, ii, present.to(F64)) > 0
    lse = m / tau + ls
    rest, erest = lse, ea + 4 * U * (m / tau).abs() + 2 * U * ls
    estat = torch.cat([erest, erest], 1)
    eq = ea + 5 * U * _finite(d).abs() + 10 * U
    grad, egrad = q - mass, q * eq + emass
    late = 6 * U * (lse.abs() + ls) * torch.ones_like(q) * q
    if tlse is not None:
        pr = (1 - p.sum(-1, keepdim=True)).clamp(min=0)
        epr = (K + _finite(t).abs().amax(-1, keepdim=True)) * 2.0 ** -51
        mr, dr, lsr, er = _states(z.masked_fill(inside, -math.inf), tau)
        below = torch.where(mr > -math.inf, (m - mr) / tau, torch.zeros_like(m))
        lqr = torch.where(mr > -math.inf, lsr - ls - below, torch.full_like(m, -math.inf))
        qr = torch.exp(lqr)
        r = torch.exp(dr - lsr)
        term = torch.where(pr > 0, pr * (pr.log() - lqr), torch.zeros_like(pr)).squeeze(1)
        loss = loss + term
        eterm = pr * (ea + er + 6 * U * (below + ls + lsr) + 16 * U * _finite(lqr).abs()) + \
            (epr + 2 * U * pr) * (1 + _finite(pr.log()).abs() + _finite(lqr).abs())
        eloss = eloss + eterm.squeeze(1) + 16 * U * _finite(term).abs()
        rest = torch.where(mr > -math.inf, mr / tau + lsr, torch.full_like(mr, -math.inf))
        estat = torch.cat([estat[:, :1], er + 4 * U * _finite(mr / tau).abs() + 2 * U * lsr], 1)
        grad = torch.where(inside, grad, r * (qr - pr))
        outside = r * ((qr + pr) * (ea + er + 5 * U * _finite(dr).abs() + 10 * U) + qr * 5 * U * below + epr)
        egrad = torch.where(inside, egrad, outside)
        late = torch.where(inside, late, r * (qr + pr) * 6 * U * (lse.abs() + _finite(rest).abs() + ls + lsr))
    stats = torch.cat([lse, rest], 1)
    stats = torch.where(torch.isfinite(stats), stats.clamp(-FLT_MAX, FLT_MAX), stats)
    off = torch.where(any_, torch.full((N,), -math.inf, dtype=F64, device=S.device), torch.zeros(N, dtype=F64, device=S.device))
    stats = torch.where(on[:, None], stats, off[:, None])
    # (past 1024 the stats are not used)
    used = ((stats.abs() <= 1024) | ~torch.isfinite(stats)).all(-1, keepdim=True)
    late = torch.where(used, late, torch.zeros_like(late))
    weight = (w.to(F64) if w is not None else torch.ones(N, dtype=F64, device=S.device))[:, None] / tau
    gate = lambda a: torch.where(on[:, None], a * weight, torch.zeros_like(a))
    # (exponentials below 2^-126 are 0)
    loss = torch.where(loss > FLT_MAX, torch.full_like(loss, math.inf), loss)
    return ((torch.where(on, loss, torch.zeros_like(loss)), eloss), (stats, torch.where(torch.isfinite(estat), estat, torch.zeros_like(estat))),
            (gate(grad), gate(egrad) + 2.0 ** -125 * (1 + weight), gate(late)))


def _check(S, idx, val, tau, tl, w, gdtype=None):
    tau = f32(tau)
    gd = S.dtype if gdtype is None else gdtype
    (wl, el), (ws, es), (wg, eg, late) = _want(S, idx, val, tau, tl, w)
    loss, stats, grad = ds.distill_loss(S, idx, val, temperature=tau, teacher_lse=tl, weight=w, grad=True, grad_dtype=gdtype)
    ref.assert_close(loss, wl, el, "loss")
    ref.assert_close(stats, ws, es, "stats")
    rounding = 1.01 * ref.HALF[gd] * wg.abs() + ref.TINY[gd]
    ref.assert_close(grad, wg, 1.01 * eg + rounding, "gradient")
    alone = ds.distill_loss(S, idx, val, temperature=tau, teacher_lse=tl)
    ref.assert_close(alone[0], wl, el, "loss alone")
    g = torch.ones(len(S), device="cuda") if w is None else w
    back = ds.distill_loss_backward(S, idx, val, stats, g, temperature=tau, teacher_lse=tl, grad_dtype=gdtype)
    ref.assert_close(back, wg, 1.01 * (eg + late) + rounding, "gradient alone")
    return loss, stats, grad, back


def _case(N, V, K, dtype, seed, tau=1.0, share=0.7):
    """Student rows, and a teacher whose kept entries carry `share` of its mass."""
    S = ref.logits(N, V, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)]).to(torch.int32)
    val = torch.empty((N, K), device="cuda").normal_(0, 2, generator=g)
    tl = torch.logsumexp(val / f32(tau), -1) - math.log(share)
    w = torch.rand(N, generator=g, device="cuda") + 0.1
    return S, idx, val, tl, w


MASKS = [-math.inf, -1e4, -3e3, -1e9, "lowest"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [1.0, 0.5])
@pytest.mark.parametrize("mask", MASKS)
def test_entries_outside_the_kept_ones_masked(dtype, tau, mask):
    fill = torch.finfo(dtype).min if mask == "lowest" else mask
    if abs(fill) > torch.finfo(dtype).max and fill != -math.inf:
        pytest.skip("not a value of the type")
    for N, V, K in ((4, 5003, 8), (2, 151936, 64)):
        S, idx, val, tl, w = _case(N, V, K, dtype, 7, tau)
        kept = S.gather(1, idx.long())
        S[:] = fill
        S[1, : V // 2] = -math.inf                 # masks of two kinds
        S.scatter_(1, idx.long(), kept)
        _check(S, idx, val, tau, tl, w)
        _check(S, idx, val, tau, None, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [1.0, 0.5, 0.01, 3.0])
@pytest.mark.parametrize("level", [1e9, -1e9, 3000.0, -3000.0, "lowest"])
def test_rows_far_from_zero(dtype, tau, level):
    level = torch.finfo(dtype).min if level == "lowest" else level
    if abs(level) > torch.finfo(dtype).max:
        level = math.copysign(6e4, level)
    S, idx, val, tl, w = _case(3, 100, 50, dtype, 3, tau)
    S[0] = level                                   # one value, half of its entries kept
    S[1] += level                                  # what of the row the type leaves
    if level < -1e5:
        S[1, ::3] = 0.0
    _check(S, idx, val, tau, tl, w)
    _check(S, idx, val, tau, None, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("gdtype", [None, torch.bfloat16])
def test_masked_empty_absent_and_repeated(dtype, tail, gdtype):
    if gdtype is not None and dtype != torch.float32:
        pytest.skip("the gradient has the logits' type")
    N, V, K = 10, 1500, 8
    S, i, v, t, w = _case(N, V, K, dtype, 11)
    S[0] = -math.inf                               # nothing left in the student
    S[1, ::2] = -math.inf
    i[1] = torch.arange(1, 2 * K, 2, dtype=torch.int32, device="cuda")
    S[2] = torch.finfo(dtype).min                  # uniform
    S[3, 5:] = torch.finfo(dtype).min              # all but entries that are kept
    i[3] = torch.arange(K, dtype=torch.int32, device="cuda").clamp(max=4)
    i[4, 3:] = -1                                  # absent entries
    i[5] = -1                                      # no teacher: the row does not count
    i[6] = i[6, 0]                                 # one index K times
    i[7, 1] = i[7, 0]
    v[8, 2] = -math.inf                            # an entry without mass
    S[9] = -math.inf                               # nothing outside the kept entries, and no mass there either
    S[9, i[9].long()] = 1.0
    t[9] = torch.logsumexp(v[9], -1) - 1e-3
    loss, _, grad, back = _check(S, i, v, 1.0, t if tail else None, w, gdtype)
    for row in (0, 5):
        assert loss[row] == 0 and (grad[row] == 0).all() and (back[row] == 0).all()


def _almost_all(kept, left, shift, tau, N, K, device="cuda"):
    """val [N, K] and teacher_lse [N] of a teacher with about `left` of its mass
    outside, and the mass that these rounded inputs leave there."""
    g = torch.Generator().manual_seed(5)
    p = torch.softmax(3.0 * torch.randn((N, K), generator=g, dtype=F64), -1) if kept == "peaked" else \
        torch.softmax(torch.log(0.5 + torch.rand((N, K), generator=g, dtype=F64)), -1)
    tl = torch.full((N,), shift, dtype=torch.float32)
    val = (tau * ((p * (1 - left)).log() + shift)).float()
    rest = 1 - torch.exp(val.to(F64) / tau - tl.to(F64)[:, None]).sum(-1)
    return val.to(device), tl.to(device), rest


LEFT = [(1e-2, 0.0), (1e-2, 12.0), (1e-4, 0.0), (1e-4, 12.0), (1e-5, 0.0), (1e-6, 0.0), (3e-7, 0.0)]


@pytest.mark.parametrize("kept", ["peaked", "spread"])
@pytest.mark.parametrize("left,shift", LEFT)
@pytest.mark.parametrize("tau", [1.0, 0.7, 3.0])
def test_teachers_that_kept_almost_all(kept, left, shift, tau):
    """The remaining mass p_r is all of the gradient outside the kept entries
    where the student has nothing there, and 1 - sum p in 32 bits is off by 2^-24
    of 1, however small p_r is."""
    N, V, K = 4, 20000, 64
    val, tl, rest = _almost_all(kept, left, shift, f32(tau), N, K)
    assert (rest > left / 4).all() and (rest < 4 * left).all()
    S = ref.logits(N, V, torch.float32, 2)
    idx = S.topk(K).indices.to(torch.int32)
    S.scatter_add_(1, idx.long(), torch.full((N, K), 60.0 * tau, device="cuda"))
    _, _, grad, back = _check(S, idx, val, tau, tl, None)
    outside = torch.ones_like(S, dtype=torch.bool).scatter_(1, idx.long(), False)
    for got in (grad, back):
        total = -(got.to(F64) * outside).sum(-1).cpu() * f32(tau)
        assert ((total - rest).abs() < 1e-4 * rest).all()
    _check(S, idx, val, tau, tl, None, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows_in_place_and_captured(dtype):
    """The rows that the gradient alone reads again, written over themselves by
    clusters of CTAs, of one wave and of several, and replayed from a graph."""
    for N, V in ((3, 40961), (700, 2049), (2, 262144)):
        S, idx, val, tl, w = _case(N, V, 24, dtype, 5)
        kept = S.gather(1, idx.long())
        S[::2] = torch.finfo(dtype).min
        S.scatter_(1, idx.long(), kept)
        _, stats, _ = ds.distill_loss(S, idx, val, teacher_lse=tl)
        want = ds.distill_loss_backward(S, idx, val, stats, w, teacher_lse=tl)
        got = S.clone()
        assert ds.distill_loss_backward(got, idx, val, stats, w, teacher_lse=tl, out=got) is got
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ds.distill_loss_backward(S, idx, val, stats, w, teacher_lse=tl)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
