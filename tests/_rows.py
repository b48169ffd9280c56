"""Plain 64-bit forms of the operators on rows of logits, and the bounds of
their rounding errors (shared by the tests; torch, any device)."""
import math

import torch

F64 = torch.float64
U = 2.0 ** -24              # half a step of float32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def logits(N, V, dtype, seed, sigma=3.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.empty((N, V), device=device).normal_(0.0, sigma, generator=g)
    x[torch.arange(N, device=device), torch.randint(0, V, (N,), generator=g, device=device)] += 8.0
    return x.to(dtype)


def base_error(V, span):
    """Relative error of a row's sum of exponentials: a lane adds V / 512 terms
    one after another (half a step each), the lanes, warps and CTAs 14 levels of
    pairs; 2^x is off by 2^-22 = 4 steps, its argument x - m and the product
    with log2 e by a step of |x - m| <= span each; 32 more for the handful of
    operations after the sum."""
    return U * (V / 512 + 14 + 4 + 3 * span + 32)


def logprobs(x, tokens, K):
    """logp, entropy, lse, top_idx, top_logp of finite or -inf rows."""
    z = x.to(F64)
    m = z.amax(-1, keepdim=True)
    none = (m == -math.inf).squeeze(-1)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s = torch.exp(z - m).sum(-1, keepdim=True)
    lse = (m + torch.log(s)).squeeze(-1)
    lse = torch.where(none, torch.full_like(lse, -math.inf), lse)
    # (not z - lse: a maximum of the type's lowest value swallows log s, in 64 bits too)
    lp = (z - m) - torch.where(none[:, None], torch.zeros_like(s), torch.log(s))
    p = torch.exp(lp)
    H = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    t = tokens.long()
    logp = lp.gather(1, t.clamp(0, x.shape[1] - 1)[:, None]).squeeze(-1)
    logp = torch.where(none, torch.full_like(logp, -math.inf), logp)
    logp = torch.where(t == -1, torch.zeros_like(logp), logp)
    logp = torch.where((t < -1) | (t >= x.shape[1]), torch.full_like(logp, math.nan), logp)
    if K == 0:
        return logp, H, lse, None, None
    order = torch.sort(z, dim=-1, descending=True, stable=True)
    idx, val = order.indices[:, :K], order.values[:, :K]
    top = lp.gather(1, idx)
    idx = torch.where(val == -math.inf, torch.full_like(idx, -1), idx)
    top = torch.where(val == -math.inf, torch.full_like(top, -math.inf), top)
    return logp, H, lse, idx.to(torch.int32), top


def logprobs_backward(x, tokens, lse, entropy, g_logp, g_entropy):
    """The gradient and the sum of its terms' sizes (for its error bound)."""
    z = x.to(F64)
    on = (lse > -math.inf)[:, None]
    m = torch.where(on, z.amax(-1, keepdim=True), torch.zeros_like(z[:, :1]))
    ls = torch.where(lse.abs()[:, None] > 1024.0, torch.log(torch.exp(z - m).sum(-1, keepdim=True)), lse.to(F64)[:, None] - m)
    d = torch.where(on, (z - m) - ls, torch.full_like(z, -math.inf))
    p = torch.exp(d)
    dd = torch.where(p > 0, d, torch.zeros_like(d))
    hit = torch.zeros_like(z)
    ok = tokens >= 0
    hit[ok, tokens[ok].long()] = 1.0
    gl = torch.where(ok, g_logp.to(F64), torch.zeros_like(lse, dtype=F64))[:, None]
    gh, H = g_entropy.to(F64)[:, None], entropy.to(F64)[:, None]
    g = torch.where(on, gl * (hit - p) - gh * p * (dd + H), torch.zeros_like(z))
    size = p * (gl.abs() + gh.abs() * (dd.abs() + H)) * (8 + 3 * dd.abs()) + hit * gl.abs()
    return g, torch.where(on, size, torch.zeros_like(z))


def distill(S, idx, val, tau, tlse, weight):
    """loss, stats, gradient [N, V] and the error bounds of loss and gradient."""
    N, V = S.shape
    z = S.to(F64) / tau
    t = val.to(F64) / tau
    present = idx >= 0
    ii = idx.long().clamp(min=0)
    t = torch.where(present, t, torch.full_like(t, -math.inf))
    any_ = (t > -math.inf).any(-1)
    norm = tlse.to(F64)[:, None] if tlse is not None else torch.where(any_, torch.logsumexp(t, -1), torch.zeros(N, dtype=F64, device=S.device))[:, None]
    lp = t - norm
    p = torch.exp(lp)
    row_on = any_ & (z.amax(-1) > -math.inf)
    lse = torch.where(row_on, torch.logsumexp(z, -1), torch.zeros(N, dtype=F64, device=S.device))
    lq = z - lse[:, None]
    q = torch.exp(lq)
    gap = torch.where(p > 0, lp - lq.gather(1, ii), torch.zeros_like(lp))
    loss = (p * gap).sum(-1)
    size = (p * gap.abs()).sum(-1)
    mass = torch.zeros_like(z).scatter_add_(1, ii, p)
    inside = torch.zeros_like(z).scatter_add_(1, ii, present.to(F64)) > 0
    grad = q - mass
    gsize = q + mass
    rest = lse
    if tlse is not None:
        pr = (1 - p.sum(-1)).clamp(min=0)
        rest = torch.logsumexp(z.masked_fill(inside, -math.inf), -1)
        lqr = rest - lse
        term = torch.where(pr > 0, pr * (pr.log() - lqr), torch.zeros_like(pr))
        loss = loss + term
        size = size + term.abs() + (1 + torch.where(pr > 0, (pr.log() - lqr).abs(), torch.zeros_like(pr)))
        r = torch.where(rest[:, None] > -math.inf, torch.exp(z - rest[:, None]), torch.zeros_like(z))
        qr = torch.exp(lqr)[:, None]
        grad = torch.where(inside, grad, r * (qr - pr[:, None]))
        gsize = torch.where(inside, gsize, r * (qr + pr[:, None] + 1))
    w = torch.ones(N, dtype=F64, device=S.device) if weight is None else weight.to(F64)
    zero = torch.zeros_like(loss)
    loss = torch.where(row_on, loss, zero)
    off = torch.where(any_, torch.full_like(zero, -math.inf), zero)   # (an empty row's stats; 0 where it does not count)
    stats = torch.stack([torch.where(row_on, lse, off), torch.where(row_on, rest, off)], -1)
    grad = torch.where(row_on[:, None], grad * (w / tau)[:, None], torch.zeros_like(grad))
    gsize = torch.where(row_on[:, None], gsize * (w.abs() / tau)[:, None], torch.zeros_like(grad))
    return loss, stats, grad, 2 + size + lse.abs(), gsize


def assert_close(got, want, tol, what):
    """|got - want| <= tol, infinities and NaN in the same places."""
    got = got.to(F64)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    tol = torch.as_tensor(tol, dtype=F64, device=want.device).expand(want.shape)
    off = (got - want).abs()[fin] - tol[fin]
    assert not (off > 0).any(), f"{what}: off by {float((got - want).abs()[fin].max()):.3e}, {float(off.max()):.3e} too much"
