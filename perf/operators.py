"""Cases of the operators that read rows of logits and train the draft head.

The operators, as a user calls them (``import speculative_decoding_02_gb300 as ds``):

  token_logprobs            log probability of a given token in each row of logits, the row's
                            entropy and its most probable alternatives
  emitted_logprobs          the same for the tokens that a round emitted (the accepted drafts
                            and the corrected or bonus token), from the target logits
  token_logprobs_backward   the gradient of log probability and entropy
  distill_loss              Kullback-Leibler loss of a student's logits against a teacher's top
                            logits, with or without the gradient in the same call
  distill_loss_backward     that gradient for an upstream gradient known later
  markov_logits             the Markov head's logits l_k = U_k + W1[x_{k-1}] W2^T, teacher forced
  markov_head_backward      the gradients of W1 and W2 from the gradient of those logits

``run`` takes the plain torch form of each (32-bit elementary operations) or, with ``own`` set,
the framework's call.  ``exact`` restates each in 64 bits.
"""
import math

import torch

own = False

RANK = 256        # the Markov head's rank
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded position of one request: the latency of a single row
        dict(name="logprobs_single_row", op="logprobs", B=1, G=1, V=151936, K=20, dtype="f32", padded=False),
        # the tokens that a batch-128 round emitted, about 4 of 17 rows of each request
        dict(name="emitted_batch128", op="emitted", B=128, G=16, V=151936, K=20, dtype="f32", padded=False),
        # a teacher's pass over a batch of positions whose top logits are kept for distillation
        dict(name="logprobs_teacher_bf16", op="logprobs", B=2048, G=1, V=129280, K=64, dtype="bf16", padded=True),
        # policy-gradient training: log probability and entropy, the large vocabulary
        dict(name="logprobs_backward_large_vocab", op="logprobs_backward", B=640, G=1, V=262144, K=0, dtype="f32",
             padded=False),
        # one small evaluation batch: loss only
        dict(name="distill_eval_small", op="distill", B=16, G=5, V=32000, K=16, dtype="bf16", padded=True,
             tail=False, tau=2.0, ragged=False, grad=False),
        # one training step of the draft at the batch-128 point, the teacher's tail as one bucket
        dict(name="distill_step_batch128", op="distill", B=128, G=16, V=151936, K=64, dtype="f32", padded=False,
             tail=True, tau=1.0, ragged=False, grad=True),
        # bf16 logits, verified positions only (a ragged batch of the serving shape)
        dict(name="distill_step_ragged_bf16", op="distill", B=512, G=5, V=129280, K=32, dtype="bf16", padded=False,
             tail=False, tau=1.5, ragged=True, grad=True),
        # the backward pass alone, fp16 logits of an odd vocabulary (rows start off alignment)
        dict(name="distill_backward_odd_f16", op="distill_backward", B=200, G=7, V=50257, K=50, dtype="f16",
             padded=False, tail=True, tau=1.0, ragged=False),
        # the head's logits for a small training batch
        dict(name="markov_logits_small", op="markov_logits", B=16, G=4, V=4096, dtype="f32"),
        # and at the batch-128 point
        dict(name="markov_logits_batch128", op="markov_logits", B=128, G=16, V=151936, dtype="f32"),
        # the head's weight gradients for a small batch, and at the batch-128 point
        dict(name="head_backward_small", op="head_backward", B=16, G=4, V=8192),
        dict(name="head_backward_batch128", op="head_backward", B=128, G=16, V=151936),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "emitted", "logprobs_backward", "distill", "distill", "distill_backward",
                     "markov_logits", "head_backward"])
    most = 2048 * 151936
    G = rng.randint(1, 16)
    if op in ("markov_logits", "head_backward"):
        V = 8 * _log_uniform(rng, 128, 18992)
        B = _log_uniform(rng, 1, max(1, min(512, most // (G * V))))
        case = dict(op=op, B=B, G=G, V=V)
        if op == "markov_logits":
            case["dtype"] = rng.choice(["f32", "bf16"])
        return case
    V = _log_uniform(rng, 1000, 262144)
    if op in ("logprobs", "logprobs_backward"):
        G = 1
    rows = G + 1 if op == "emitted" else G
    B = _log_uniform(rng, 1, max(1, min(4096, most // (rows * V))))
    case = dict(op=op, B=B, G=G, V=V, dtype="f32" if op == "emitted" else rng.choice(["f32", "bf16", "f16"]),
                padded=rng.random() < 0.3)
    if op in ("logprobs", "emitted"):
        case["K"] = rng.choice([0, 1, 5, 20, 64, rng.randint(1, 128)])
    elif op == "logprobs_backward":
        case["K"] = 0
    else:
        case |= dict(K=rng.choice([1, 8, 32, 64, rng.randint(1, 128)]), tail=rng.random() < 0.5,
                     tau=rng.choice([1.0, 1.0, 2.0, round(rng.uniform(0.7, 4.0), 2)]), ragged=rng.random() < 0.4)
        if op == "distill":
            case["grad"] = rng.random() < 0.7
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(B, most, keep):
    """B accepted prefixes of at most `most` positions, each of which goes on with probability `keep`: the
    quantiles of that law, so that their sum is the same for every seed."""
    return [min(most, int(math.log(1.0 - (i + 0.5) / B) / math.log(keep))) for i in range(B)]


def _shuffled_lengths(B, most, keep, gen):
    n = torch.tensor(_lengths(B, most, keep), dtype=torch.int32, device="cuda")
    return n[torch.randperm(B, generator=gen, device="cuda")].contiguous()


def _normal(shape, sigma, gen, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen).to(dtype)


def _tokens(shape, V, gen):
    """Token ids with frequent ones among them (the density falls with the id)."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    return (u * u * u * V).to(torch.int32).clamp_(max=V - 1)


def _logits(N, V, dtype, padded, gen):
    """Rows as a language model gives them: noise with one likelier token; `padded` masks the vocabulary's
    unused last entries."""
    x = _normal((N, V), 3.0, gen)
    peak = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
    x.scatter_add_(1, peak, torch.full((N, 1), 8.0, device="cuda"))
    if padded:
        x[:, V - V // 50:] = -math.inf
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 17)
    op, B, G, V = case["op"], case["B"], case["G"], case["V"]
    N = B * G
    st = dict(op=op, case=case)
    if op in ("logprobs", "logprobs_backward"):
        st["logits"] = _logits(B, V, DTYPES[case["dtype"]], case["padded"], gen)
        st["tokens"] = _tokens((B,), V - V // 50, gen)
        st["K"] = case["K"]
        if op == "logprobs_backward":
            z = st["logits"].float()
            st["lse"] = torch.logsumexp(z, -1)
            z -= st["lse"][:, None]
            st["entropy"] = -torch.where(z > -math.inf, z.exp() * z, torch.zeros_like(z)).sum(-1)
            st["g_logp"] = _normal((B,), 1.0, gen)
            st["g_entropy"] = _normal((B,), 0.01, gen)
    elif op == "emitted":
        st["logits"] = _logits(B * (G + 1), V, DTYPES[case["dtype"]], case["padded"], gen).view(B, G + 1, V)
        st["x"] = _tokens((B, G), V - V // 50, gen)
        st["n"] = _shuffled_lengths(B, G, 0.75, gen)
        st["tok"] = _tokens((B,), V - V // 50, gen)
        st["K"] = case["K"]
    elif op in ("distill", "distill_backward"):
        S = _logits(N, V, torch.float32, case["padded"], gen)
        top = (S + _normal((N, V), 1.0, gen)).topk(case["K"])
        st["logits"] = S.to(DTYPES[case["dtype"]]).view(B, G, V)
        st["top_idx"] = top.indices.to(torch.int32).view(B, G, -1)
        st["top_val"] = top.values.view(B, G, -1)
        st["tau"] = case["tau"]
        # the teacher's whole mass: its K best entries carry 40 to 95 % of it
        share = 0.4 + 0.55 * torch.rand((N,), generator=gen, device="cuda")
        st["teacher_lse"] = (torch.logsumexp(top.values / case["tau"], -1) - share.log()).view(B, G) if case["tail"] else None
        k = torch.arange(G, device="cuda", dtype=torch.float32)
        st["weight"] = torch.exp(-k / G).expand(B, G).contiguous()
        st["rows"] = _shuffled_lengths(B, G, 0.8, gen) if case["ragged"] else None
        st["grad"] = case.get("grad", True)
        if op == "distill_backward":
            _, st["stats"], _ = _plain_distill(st, False)
    else:
        dt = torch.bfloat16
        st["W1"] = _normal((V, RANK), 0.02, gen, dt)
        st["W2"] = _normal((V, RANK), 0.02, gen, dt)
        st["anchor"] = _tokens((B,), V, gen)
        st["x"] = _tokens((B, G), V, gen)
        if op == "markov_logits":
            st["U"] = _normal((B, G, V), 3.0, gen)
            st["dtype"] = DTYPES[case["dtype"]]
        else:
            # the gradient that the losses above leave: a softmax less the teacher's few entries
            d = torch.softmax(_normal((N, V), 3.0, gen), -1)
            hit = torch.randint(0, V, (N, min(32, V)), generator=gen, device="cuda")
            d.scatter_add_(1, hit, -torch.softmax(_normal(hit.shape, 2.0, gen), -1))
            st["dlogits"] = d.to(dt).view(B, G, V)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _softmax_parts(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m)
    s = e.sum(-1, keepdim=True)
    return m, e, s


def _top(z, K):
    """The K largest of each row, largest first, equal ones by index: one sortable key per entry."""
    bits = (z + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    idx = torch.arange(z.shape[-1], device=z.device, dtype=torch.int64)
    key = torch.topk((order << 32) + (0xFFFFFFFF - idx), K).values
    return 0xFFFFFFFF - (key & 0xFFFFFFFF)


def _plain_logprobs(z, tokens, K):
    z = z.float()
    m, e, s = _softmax_parts(z)
    lse = (m + torch.log(s)).squeeze(-1)
    d = z - lse[:, None]
    entropy = -torch.where(e > 0, (e / s) * d, torch.zeros_like(d)).sum(-1)
    logp = d.gather(1, tokens.long()[:, None]).squeeze(-1)
    if K == 0:
        return logp, entropy, lse, None, None
    top = _top(z, K)
    top_logp = d.gather(1, top)
    top = torch.where(top_logp > -math.inf, top, torch.full_like(top, -1))
    return logp, entropy, lse, top.to(torch.int32), top_logp


def _plain_emitted(T, x, n, tok, K):
    B, R, V = T.shape
    j = torch.arange(R, device=T.device)
    live = (j[None, :] <= n[:, None]).view(-1)
    tokens = torch.where(j[None, :] < n[:, None], torch.cat([x, x[:, :1]], 1), tok[:, None]).view(-1)
    got = _plain_logprobs(T.view(-1, V)[live], tokens[live], K)
    whole = []
    for v, fill in zip(got, (0, 0, 0, -1, -math.inf)):
        if v is None:
            whole.append(None)
            continue
        w = torch.full((B * R, *v.shape[1:]), fill, dtype=v.dtype, device=v.device)
        w[live] = v
        whole.append(w.view(B, R, *v.shape[1:]))
    return tuple(whole)


def _plain_logprobs_backward(logits, tokens, lse, entropy, g_logp, g_entropy):
    d = logits.float() - lse[:, None]
    p = torch.exp(d)
    g = -p * (g_logp[:, None] + g_entropy[:, None] * torch.where(p > 0, d + entropy[:, None], torch.zeros_like(d)))
    g.scatter_add_(1, tokens.long()[:, None], g_logp[:, None])
    return g.to(logits.dtype)


def _plain_distill(st, grad):
    S = st["logits"]
    B, G, V = S.shape
    K, inv = st["top_idx"].shape[-1], 1.0 / st["tau"]
    live = slice(None)
    if st["rows"] is not None:
        live = (torch.arange(G, device=S.device)[None, :] < st["rows"][:, None]).view(-1)
    z = S.view(-1, V)[live].float() * inv
    idx = st["top_idx"].view(-1, K)[live].long()
    t = st["top_val"].view(-1, K)[live].double() * inv
    m, e, s = _softmax_parts(z)
    lse = m + torch.log(s)
    tail = st["teacher_lse"] is not None
    logp = t - (st["teacher_lse"].view(-1)[live].double()[:, None] if tail else torch.logsumexp(t, -1, keepdim=True))
    p = torch.exp(logp)
    loss = (p * (logp - (z.gather(1, idx) - lse))).sum(-1, keepdim=True)
    lse_rest, factor = lse, None
    if tail:
        p_rest = (1.0 - p.sum(-1, keepdim=True)).clamp_(min=0.0)
        lse_rest = m + torch.log(e.scatter(1, idx, 0.0).sum(-1, keepdim=True))
        loss = loss + torch.where(p_rest > 0, p_rest * (p_rest.log() - (lse_rest - lse)), torch.zeros_like(p_rest))
        factor = (1.0 - p_rest * torch.exp(lse - lse_rest)).float()
    out_loss = torch.zeros(B * G, device=S.device)
    out_stats = torch.zeros(B * G, 2, device=S.device)
    out_loss[live] = loss.float().squeeze(-1)
    out_stats[live] = torch.cat([lse, lse_rest], 1)
    dl = None
    if grad:
        w = (st["weight"].view(-1)[live] * inv)[:, None]
        q = e / s
        g = q * factor * w if tail else q * w
        g.scatter_(1, idx, (q.gather(1, idx) - p.float()) * w)
        dl = torch.zeros(B * G, V, dtype=S.dtype, device=S.device)
        dl[live] = g.to(S.dtype)
        dl = dl.view(B, G, V)
    return out_loss.view(B, G), out_stats.view(B, G, 2), dl


def _previous(st):
    return torch.cat([st["anchor"][:, None], st["x"][:, :-1]], 1).reshape(-1).long()


def _plain_markov_logits(st):
    U = st["U"]
    bias = st["W1"][_previous(st)].float() @ st["W2"].float().T
    return (U + bias.view(U.shape)).to(st["dtype"])


def _plain_head_backward(st):
    prev, W1 = _previous(st), st["W1"]
    d = st["dlogits"].view(-1, W1.shape[0]).float()
    dW2 = d.T @ W1[prev].float()
    dW1 = torch.zeros(W1.shape, device=d.device).index_add_(0, prev, d @ st["W2"].float())
    return dW1, dW2


def run(st):
    op = st["op"]
    if own:
        import speculative_decoding_02_gb300 as ds

        if op == "logprobs":
            return ds.token_logprobs(st["logits"], st["tokens"], top_k=st["K"])
        if op == "emitted":
            return ds.emitted_logprobs(st["logits"], st["x"], st["n"], st["tok"], top_k=st["K"])
        if op == "logprobs_backward":
            return ds.token_logprobs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"], st["g_logp"],
                                              st["g_entropy"])
        if op == "distill":
            return ds.distill_loss(st["logits"], st["top_idx"], st["top_val"], temperature=st["tau"],
                                   teacher_lse=st["teacher_lse"], weight=st["weight"], rows=st["rows"],
                                   grad=st["grad"])
        if op == "distill_backward":
            return ds.distill_loss_backward(st["logits"], st["top_idx"], st["top_val"], st["stats"], st["weight"],
                                            temperature=st["tau"], teacher_lse=st["teacher_lse"], rows=st["rows"])
        if op == "markov_logits":
            return ds.markov_logits(st["U"], st["W1"], st["W2"], st["anchor"], st["x"], dtype=st["dtype"])
        return ds.markov_head_backward(st["dlogits"], st["W1"], st["W2"], st["anchor"], st["x"])
    if op == "logprobs":
        return _plain_logprobs(st["logits"], st["tokens"], st["K"])
    if op == "emitted":
        return _plain_emitted(st["logits"], st["x"], st["n"], st["tok"], st["K"])
    if op == "logprobs_backward":
        return _plain_logprobs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"], st["g_logp"],
                                        st["g_entropy"])
    if op == "distill":
        return _plain_distill(st, st["grad"])
    if op == "distill_backward":
        return _plain_distill(st, True)[2]
    if op == "markov_logits":
        return _plain_markov_logits(st)
    return _plain_head_backward(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, B, G, V = case["op"], case["B"], case["G"], case["V"]
    K = case.get("K", 0)
    if op in ("markov_logits", "head_backward"):
        N, weights = B * G, 2 * RANK * V
        gathered = 2 * RANK * min(N, V)
        if op == "markov_logits":
            out = 4 if case["dtype"] == "f32" else 2
            return {"bytes": N * V * (4 + out) + weights + gathered, "flops": 2.0 * N * V * RANK}
        return {"bytes": 2 * N * V + weights + gathered + 2 * 4 * RANK * V, "flops": 4.0 * N * V * RANK}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "emitted":
        rows = sum(n + 1 for n in _lengths(B, G, 0.75))
    else:
        rows = sum(_lengths(B, G, 0.8)) if case.get("ragged") else B * G
    if op in ("logprobs", "emitted"):
        return {"bytes": rows * (V * size + 4) + B * (G + 1 if op == "emitted" else 1) * (12 + 8 * K),
                "flops": 5.0 * rows * V}
    if op == "logprobs_backward":
        return {"bytes": rows * (2 * V * size + 20), "flops": 5.0 * rows * V}
    teacher = rows * (8 * K + 8)
    if op == "distill_backward":
        return {"bytes": rows * V * size + B * G * V * size + teacher, "flops": 4.0 * rows * V}
    if case["grad"]:
        return {"bytes": rows * V * size + B * G * (V * size + 12) + teacher, "flops": 6.0 * rows * V}
    return {"bytes": rows * V * size + B * G * 12 + teacher, "flops": 4.0 * rows * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(z, tokens, K):
    z = z.to(torch.float64)
    lse = torch.logsumexp(z, -1)
    logp = z.gather(1, tokens.long().unsqueeze(1)).squeeze(1) - lse
    lp = torch.log_softmax(z, -1)
    entropy = torch.special.entr(lp.exp()).sum(-1)
    if K == 0:
        return [logp, entropy, lse, None, None]
    return [logp, entropy, lse, None, lp.topk(K).values]


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "logprobs":
        return tuple(_exact_rows(st["logits"], st["tokens"], st["K"]))
    if op == "emitted":
        T, n = st["logits"], st["n"].tolist()
        B, R, V = T.shape
        want = [torch.zeros(B, R, dtype=f64, device=T.device) for _ in range(3)]
        want += [None, None if st["K"] == 0 else torch.full((B, R, st["K"]), -math.inf, dtype=f64, device=T.device)]
        for b in range(B):
            tokens = torch.cat([st["x"][b, :n[b]], st["tok"][b:b + 1]])
            for w, v in zip(want, _exact_rows(T[b, :n[b] + 1], tokens, st["K"])):
                if w is not None:
                    w[b, :n[b] + 1] = v
        return tuple(want)
    if op == "logprobs_backward":
        z = st["logits"].to(f64)
        lp = z - st["lse"].to(f64).unsqueeze(1)
        p = lp.exp()
        grad_entropy = torch.special.entr(p) - p * st["entropy"].to(f64).unsqueeze(1)
        grad = st["g_entropy"].to(f64).unsqueeze(1) * grad_entropy - st["g_logp"].to(f64).unsqueeze(1) * p
        at = torch.arange(z.shape[0], device=z.device)
        grad[at, st["tokens"].long()] += st["g_logp"].to(f64)
        return grad
    if op in ("distill", "distill_backward"):
        S = st["logits"]
        B, G, V = S.shape
        N, tau = B * G, st["tau"]
        z = S.reshape(N, V).to(f64) / tau
        idx = st["top_idx"].reshape(N, -1).long()
        t = st["top_val"].reshape(N, -1).to(f64) / tau
        on = torch.ones(N, dtype=torch.bool, device=S.device)
        if st["rows"] is not None:
            on = (torch.arange(G, device=S.device).unsqueeze(0) < st["rows"].unsqueeze(1)).reshape(N)
        lq = torch.log_softmax(z, -1)
        lse = torch.logsumexp(z, -1)
        inside = torch.zeros(N, V, dtype=torch.bool, device=S.device).scatter_(1, idx, True)
        if st["teacher_lse"] is None:
            lp = torch.log_softmax(t, -1)
            loss = (lp.exp() * (lp - lq.gather(1, idx))).sum(-1)
            rest = lse
            grad = lq.exp()
        else:
            lp = t - st["teacher_lse"].reshape(N, 1).to(f64)
            p_rest = 1 - lp.exp().sum(-1)
            rest = torch.logsumexp(z.masked_fill(inside, -math.inf), -1)
            loss = (lp.exp() * (lp - lq.gather(1, idx))).sum(-1) + p_rest * (p_rest.log() - (rest - lse))
            grad = lq.exp()
            grad -= torch.where(inside, 0.0, p_rest.unsqueeze(1) * torch.exp(z - rest.unsqueeze(1)))
        grad.scatter_add_(1, idx, -lp.exp())
        grad *= (st["weight"].reshape(N).to(f64) / tau * on).unsqueeze(1)
        if op == "distill_backward":
            return grad.view(B, G, V)
        stats = torch.where(on.unsqueeze(1), torch.stack([lse, rest], 1), 0.0)
        return (torch.where(on, loss, 0.0).view(B, G), stats.view(B, G, 2),
                grad.view(B, G, V) if case["grad"] else None)
    before = torch.cat([st["anchor"].unsqueeze(1), st["x"]], 1)[:, :-1].flatten().long()
    E, W2 = st["W1"].to(f64)[before], st["W2"].to(f64)
    if op == "markov_logits":
        return st["U"].to(f64) + torch.einsum("nr,vr->nv", E, W2).view(st["U"].shape)
    d = st["dlogits"].to(f64).flatten(0, 1)
    dW1 = torch.zeros(W2.shape, dtype=f64, device=d.device)
    dW1.index_put_((before,), torch.einsum("nv,vr->nr", d, W2), accumulate=True)
    return dW1, torch.einsum("nv,nr->vr", d, E)
