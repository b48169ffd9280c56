"""Cases of the operators that train a draft from its hidden states.

The operators, as a user calls them (``import speculative_decoding_02_gb300 as ds``):

  linear_cross_entropy           softmax cross entropy of hidden states under an output head W [V, D],
                                 taken in pieces of the vocabulary, so that the logits h W^T are never kept
  linear_cross_entropy_backward  its gradients: of the hidden states, of the head, or of both
  newton_schulz                  an update orthogonalised by Newton-Schulz products, as the Muon
                                 optimiser takes it

``run`` takes the plain torch form of each (32-bit elementary operations) or, with ``own`` set,
the framework's call.  ``exact`` restates each in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


def listed():
    return [
        # the score of one token of one request under the target's head: the latency of a single row
        dict(name="loss_single_row", op="loss", B=1, G=1, V=151936, D=2560, dtype="bf16", ragged=False, masked=0.0),
        # a small evaluation batch of drafts of different lengths
        dict(name="loss_eval_small", op="loss", B=16, G=5, V=32000, D=1024, dtype="f16", ragged=True, masked=0.0),
        # the loss of one draft batch at the batch-128 point
        dict(name="loss_batch128", op="loss", B=128, G=16, V=151936, D=2560, dtype="bf16", ragged=False, masked=0.0),
        # an odd vocabulary, an odd number of positions, a prompt's positions without a target among them
        dict(name="loss_odd_f16", op="loss", B=1003, G=1, V=50257, D=1032, dtype="f16", ragged=False, masked=0.3),
        # both gradients of a small batch
        dict(name="backward_small", op="backward", B=16, G=4, V=8192, D=512, dtype="bf16", ragged=False, masked=0.0,
             dh=True, dW=True, zloss=False),
        # the draft's own step: the head is the target's and stays as it is, only the hidden states learn
        dict(name="backward_frozen_batch128", op="backward", B=128, G=16, V=151936, D=2560, dtype="bf16", ragged=False,
             masked=0.0, dh=True, dW=False, zloss=False),
        # both gradients for the serving shape with its verified positions only
        dict(name="backward_ragged_serving", op="backward", B=512, G=5, V=129280, D=4096, dtype="bf16", ragged=True,
             masked=0.0, dh=True, dW=True, zloss=False),
        # a whole step, the loss and then both gradients, with a penalty on the log-sum-exp, the large vocabulary
        dict(name="step_large_vocab", op="step", B=64, G=8, V=262144, D=3840, dtype="bf16", ragged=False, masked=0.0,
             dh=True, dW=True, zloss=True),
        # one small square weight: a chain of products bound by latency
        dict(name="orthogonal_small", op="orthogonal", m=256, n=256, dtype="f32"),
        # odd sizes, a bf16 momentum
        dict(name="orthogonal_odd_bf16", op="orthogonal", m=1000, n=777, dtype="bf16"),
        # a square weight of the serving shape's hidden size
        dict(name="orthogonal_square", op="orthogonal", m=4096, n=4096, dtype="f32"),
        # the gradient of one weight of the Markov head: rank 256, a row for each token
        dict(name="orthogonal_head", op="orthogonal", m=151936, n=256, dtype="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "backward", "backward", "step", "orthogonal", "orthogonal"])
    if op == "orthogonal":
        dtype = rng.choice(["f32", "bf16", "f16"])
        if rng.random() < 0.25:
            case = dict(op=op, m=_log_uniform(rng, 4096, 200000), n=_log_uniform(rng, 16, 256), dtype=dtype)
        else:
            case = dict(op=op, m=_log_uniform(rng, 16, 4096), n=_log_uniform(rng, 16, 4096), dtype=dtype)
        if rng.random() < 0.3:
            case["m"], case["n"] = case["n"], case["m"]
        return case
    V, D = _log_uniform(rng, 1000, 262144), 8 * _log_uniform(rng, 8, 512)
    most = 2560 * 129280 * 4096 // (4 if op == "step" else 3)
    G = rng.randint(1, 16)
    B = _log_uniform(rng, 1, max(1, min(2048, most // (G * V * D))))
    case = dict(op=op, B=B, G=G, V=V, D=D, dtype=rng.choice(["bf16", "bf16", "f16"]), ragged=B > 7 and rng.random() < 0.4,
                masked=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]))
    if op != "loss":
        dh = rng.random() < 0.85
        case |= dict(dh=dh, dW=not dh or rng.random() < 0.6, zloss=rng.random() < 0.3)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(B, most, keep):
    """B prefixes of at most `most` positions, each of which goes on with probability `keep`: the quantiles of
    that law, so that their sum is the same for every seed."""
    return [min(most, int(math.log(1.0 - (i + 0.5) / B) / math.log(keep))) for i in range(B)]


def _normal(shape, sigma, gen, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 29)
    dtype = DTYPES[case["dtype"]]
    st = dict(op=case["op"])
    if case["op"] == "orthogonal":
        # a momentum: a few strong directions, many weak ones, noise
        m, n = case["m"], case["n"]
        k = min(32, m, n)
        strong = _normal((m, k), 1.0, gen) * torch.exp(-0.2 * torch.arange(k, device="cuda"))
        st["update"] = (1e-3 * (strong @ _normal((k, n), 1.0, gen) + _normal((m, n), 0.3, gen))).to(dtype)
        return st
    B, G, V, D = case["B"], case["G"], case["V"], case["D"]
    # hidden states point to the head's row of their token, which has a logit of 0 to 12 in noise of 2; frequent
    # tokens come often
    u = torch.rand((B, G), generator=gen, device="cuda", dtype=torch.float64)
    tokens = (u * u * u * V).to(torch.int32).clamp_(max=V - 1)
    st["W"] = _normal((V, D), 2.0 / math.sqrt(D), gen, dtype)
    sure = 12.0 * torch.rand((B, G, 1), generator=gen, device="cuda")
    st["h"] = (_normal((B, G, D), 1.0, gen) + sure / 4.0 * st["W"][tokens.long()].float()).to(dtype)
    gone = torch.randperm(B * G, generator=gen, device="cuda").view(B, G) < int(case["masked"] * B * G)
    st["tokens"] = torch.where(gone, -1, tokens).to(torch.int32)
    st["rows"] = None
    if case["ragged"]:
        n = torch.tensor(_lengths(B, G, 0.8), dtype=torch.int32, device="cuda")
        st["rows"] = n[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    if case["op"] != "loss":
        k = torch.arange(G, device="cuda", dtype=torch.float32)
        st["g_loss"] = torch.exp(-k / G).expand(B, G).contiguous()
        st["g_lse"] = _normal((B, G), 1e-3, gen) if case["zloss"] else None
        st["dh"], st["dW"] = case["dh"], case["dW"]
    if case["op"] == "backward":
        st["lse"] = _plain_loss(st)[1]
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _live(st):
    live = st["tokens"] >= 0
    if st["rows"] is not None:
        live &= torch.arange(live.shape[1], device=live.device)[None, :] < st["rows"][:, None]
    return live


def _plain_logits(st, live):
    return st["h"][live].float() @ st["W"].float().T


def _plain_loss(st):
    live = _live(st)
    z = _plain_logits(st, live)
    m = z.amax(-1, keepdim=True)
    lse = (m + torch.log(torch.exp(z - m).sum(-1, keepdim=True))).squeeze(-1)
    loss = lse - z.gather(1, st["tokens"][live].long()[:, None]).squeeze(-1)
    out = torch.zeros(2, *live.shape, device=live.device)
    out[0, live], out[1, live] = loss, lse
    return out[0], out[1]


def _plain_backward(st, lse):
    live = _live(st)
    g = st["g_loss"][live][:, None]
    d = torch.exp(_plain_logits(st, live) - lse[live][:, None])
    d *= g if st["g_lse"] is None else g + st["g_lse"][live][:, None]
    d.scatter_add_(1, st["tokens"][live].long()[:, None], -g)
    dh = dW = None
    if st["dh"]:
        dh = torch.zeros_like(st["h"])
        dh[live] = (d @ st["W"].float()).to(dh.dtype)
    if st["dW"]:
        dW = (d.T @ st["h"][live].float()).to(st["W"].dtype)
    return dh, dW


def _plain_orthogonal(M):
    a, b, c = COEFFICIENTS
    X = M.float() if M.shape[0] <= M.shape[1] else M.float().T
    X = X / (X.square().sum().sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X if M.shape[0] <= M.shape[1] else X.T).to(torch.bfloat16).contiguous()


def run(st):
    op = st["op"]
    if own:
        import speculative_decoding_02_gb300 as ds

        if op == "orthogonal":
            return ds.newton_schulz(st["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        if op == "backward":
            return ds.linear_cross_entropy_backward(st["h"], st["W"], st["tokens"], st["lse"], st["g_loss"],
                                                    g_lse=st["g_lse"], rows=st["rows"], dh=st["dh"], dW=st["dW"])
        loss, lse = ds.linear_cross_entropy(st["h"], st["W"], st["tokens"], rows=st["rows"])
        if op == "loss":
            return loss, lse
        dh, dW = ds.linear_cross_entropy_backward(st["h"], st["W"], st["tokens"], lse, st["g_loss"], g_lse=st["g_lse"],
                                                  rows=st["rows"], dh=st["dh"], dW=st["dW"])
        return loss, lse, dh, dW
    if op == "orthogonal":
        return _plain_orthogonal(st["update"])
    if op == "backward":
        return _plain_backward(st, st["lse"])
    loss, lse = _plain_loss(st)
    if op == "loss":
        return loss, lse
    return (loss, lse, *_plain_backward(st, lse))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "orthogonal":
        small, large = sorted((case["m"], case["n"]))
        size = 4 if case["dtype"] == "f32" else 2
        # a step: the Gram matrix and its square (symmetric: one half of each), and the product with X
        return {"bytes": small * large * (size + 2.0),
                "flops": STEPS * (1.0 * small * small * large + 1.0 * small ** 3 + 2.0 * small * small * large)}
    B, G, V, D = case["B"], case["G"], case["V"], case["D"]
    rows = sum(_lengths(B, G, 0.8)) if case["ragged"] else B * G
    rows = max(1.0, rows * (1.0 - case["masked"]))
    # the products: the logits, once for the loss and (they are not kept) once for the gradients; dh; dW
    products = 1 if case["op"] == "loss" else 1 + case["dh"] + case["dW"] + (case["op"] == "step")
    size = 2.0 * (V * D + rows * D) + 4.0 * B * G
    size += 8.0 * B * G if case["op"] != "backward" else 8.0 * rows
    if case["op"] != "loss":
        size += 2.0 * (B * G * D * case["dh"] + V * D * case["dW"]) + (4.0 + 4.0 * case["zloss"]) * rows
    return {"bytes": size, "flops": 2.0 * products * rows * V * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "orthogonal":
        # on the other side than the plain form's products, a row vector's view of the same polynomial
        M = st["update"].to(f64)
        tall = M.shape[0] >= M.shape[1]
        Y = M if tall else M.mT
        Y = Y / (torch.linalg.matrix_norm(Y) + EPS)
        one = torch.eye(Y.shape[1], dtype=f64, device=Y.device)
        for _ in range(STEPS):
            S = Y.mT @ Y
            Y = Y @ (COEFFICIENTS[0] * one + S @ (COEFFICIENTS[1] * one + COEFFICIENTS[2] * S))
        return Y if tall else Y.mT.contiguous()
    B, G, D = st["h"].shape
    V = st["W"].shape[0]
    token = st["tokens"].flatten().long()
    on = token != -1
    if st["rows"] is not None:
        on &= (torch.arange(B * G, device=on.device) % G) < st["rows"].repeat_interleave(G)
    at = on.nonzero().flatten()
    h, W, t = st["h"].flatten(0, 1)[at].to(f64), st["W"].to(f64), token[at]
    logits = torch.einsum("nd,vd->nv", h, W)
    picked = logits[torch.arange(at.numel(), device=at.device), t]
    own_lse = torch.logsumexp(logits, 1)

    def whole(rows, *more):
        return torch.zeros(B * G, *more, dtype=f64, device=at.device).index_copy_(0, at, rows).view(B, G, *more)

    if case["op"] == "loss":
        return whole(own_lse - picked), whole(own_lse)
    lse = own_lse if case["op"] == "step" else st["lse"].flatten()[at].to(f64)
    down = st["g_loss"].flatten()[at].to(f64)
    up = down if st["g_lse"] is None else down + st["g_lse"].flatten()[at].to(f64)
    slope = logits.sub_(lse.unsqueeze(1)).exp_().mul_(up.unsqueeze(1))
    slope[torch.arange(at.numel(), device=at.device), t] -= down
    dh = whole(torch.einsum("nv,vd->nd", slope, W), D) if case["dh"] else None
    dW = torch.einsum("nv,nd->vd", slope, h) if case["dW"] else None
    if case["op"] == "backward":
        return dh, dW
    return whole(own_lse - picked), whole(own_lse), dh, dW
