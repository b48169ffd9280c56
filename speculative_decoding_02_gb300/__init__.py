"""Python binding of libdspark, the GB300 (sm_103a) DSpark per-round hot path.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors must be contiguous CUDA tensors on one device; outputs are
allocated with torch on that device and every call is enqueued on the current
torch stream.  If the compiled library is missing, every call raises
``DSparkError`` -- there is no CPU fallback.  Autograd does not see these calls:
their outputs require no gradient, whatever their inputs do, and the gradients
are calls of their own (the _backward forms, and distill_loss with grad).

Entry points (same names as the C ABI in include/dspark.h; the optional
arguments of markov_draft, schedule, verify and round map to the C ABI's _ex
forms):
  markov_draft, confidence, schedule, verify, round, read_status,
  acceptance_label, sts_fit, token_logprobs, emitted_logprobs,
  token_logprobs_backward, distill_loss, distill_loss_backward,
  markov_logits, markov_head_backward, linear_cross_entropy,
  linear_cross_entropy_backward, newton_schulz
head_status is the word in which the last five record errors without a workspace.
"""
import ctypes
import functools
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libdspark.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE, ERR_NONFINITE = range(7)
F32, BF16, F16 = 0, 1, 2
SCHED_FIXED, SCHED_GREEDY, SCHED_TOPK = 0, 1, 2
EARLY_TARGET_STATS, ADVANCE_ROUND, TARGET_STATS_FROM_VERIFY, SCRATCH_FROM_DRAFT, GATED_STATES = 1, 2, 4, 8, 16
ALL_ROW_STATS = 32
CHAIN_TARGET_STATS = 64


class DSparkError(RuntimeError):
    def __init__(self, code, where=""):
        self.code = code
        msg = _strerror(code) if _lib is not None else f"status {code}"
        super().__init__(f"{where}: {msg} (status {code})" if where else msg)


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise DSparkError(ERR_CUDA, f"libdspark is not built ({LIB_PATH} missing); run "
                                    f"`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    L.dspark_workspace_size.argtypes = [i32, i32, i32]
    L.dspark_workspace_size.restype = sz
    L.dspark_markov_draft.argtypes = [vp, vp, vp, i32, vp, i32, i32, i32, i32, u64, u64, vp, vp, vp, vp, sz, vp]
    L.dspark_markov_draft.restype = i32
    L.dspark_markov_draft_ex.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, u64, u64, vp, vp, vp, vp, vp,
                                         sz, vp]
    L.dspark_markov_draft_ex.restype = i32
    L.dspark_gated_markov_draft.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, u64, u64, vp, vp,
                                            vp, vp, vp, sz, vp]
    L.dspark_gated_markov_draft.restype = i32
    L.dspark_confidence.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    L.dspark_confidence.restype = i32
    L.dspark_schedule.argtypes = [vp, i32, i32, vp, i32, i32, u64, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_schedule.restype = i32
    L.dspark_schedule_ex.argtypes = [vp, i32, i32, vp, i32, i32, u64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_schedule_ex.restype = i32
    L.dspark_verify.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, u64, u64, vp, vp,
                                vp, sz, vp]
    L.dspark_verify.restype = i32
    L.dspark_verify_ex.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, u64, u64, vp,
                                   ctypes.c_uint, vp, vp, vp, sz, vp]
    L.dspark_verify_ex.restype = i32
    L.dspark_acceptance_label.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp,
                                          ctypes.c_size_t, vp]
    L.dspark_acceptance_label.restype = i32
    L.dspark_acceptance_label_ex.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_uint,
                                             vp, vp, ctypes.c_size_t, vp]
    L.dspark_acceptance_label_ex.restype = i32
    L.dspark_sts_workspace_size.argtypes = [i32, i32, i32]
    L.dspark_sts_workspace_size.restype = sz
    L.dspark_sts_fit.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, sz, vp]
    L.dspark_sts_fit.restype = i32
    L.dspark_round.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, i32,
                               vp, u64, u64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_round.restype = i32
    L.dspark_round_ex.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, i32,
                                  vp, u64, u64, vp, ctypes.c_uint, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_round_ex.restype = i32
    L.dspark_draft_schedule.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32,
                                        i32, vp, u64, u64, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_draft_schedule.restype = i32
    L.dspark_draft_schedule_ex.argtypes = [vp, vp, vp, vp, i32, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp,
                                           i32, i32, vp, u64, u64, vp, ctypes.c_uint, vp, vp, vp, vp, vp, vp, vp,
                                           vp, sz, vp]
    L.dspark_draft_schedule_ex.restype = i32
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.dspark_token_logprobs.argtypes = [vp, i32, i64, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.dspark_token_logprobs.restype = i32
    L.dspark_emitted_logprobs.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.dspark_emitted_logprobs.restype = i32
    L.dspark_token_logprobs_backward.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp]
    L.dspark_token_logprobs_backward.restype = i32
    L.dspark_head_workspace_size.argtypes = [i32, i32, i32]
    L.dspark_head_workspace_size.restype = sz
    L.dspark_markov_logits.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp, sz, vp]
    L.dspark_markov_logits.restype = i32
    L.dspark_markov_head_backward.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_markov_head_backward.restype = i32
    L.dspark_markov_head_backward_ex.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.dspark_markov_head_backward_ex.restype = i32
    L.dspark_distill_loss.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp, vp, vp, i32, vp]
    L.dspark_distill_loss.restype = i32
    L.dspark_distill_loss_backward.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp,
                                               i32, vp]
    L.dspark_distill_loss_backward.restype = i32
    L.dspark_linear_ce_workspace_size.argtypes = [i32, i32, i32, i32]
    L.dspark_linear_ce_workspace_size.restype = sz
    L.dspark_linear_cross_entropy.argtypes = [vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.dspark_linear_cross_entropy.restype = i32
    L.dspark_linear_cross_entropy_backward.argtypes = [vp, i64, vp, i64, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp,
                                                       vp, vp, vp, sz, vp]
    L.dspark_linear_cross_entropy_backward.restype = i32
    L.dspark_newton_schulz_workspace_size.argtypes = [i32, i32]
    L.dspark_newton_schulz_workspace_size.restype = sz
    L.dspark_newton_schulz.argtypes = [vp, i32, i64, i32, i32, i32, f32, f32, f32, f32, vp, vp, vp, sz, vp]
    L.dspark_newton_schulz.restype = i32
    L.dspark_read_status.argtypes = [vp, ctypes.POINTER(i32), vp]
    L.dspark_read_status.restype = i32
    L.dspark_selftest_wait_timeout.argtypes = [i32, vp, sz, vp]
    L.dspark_selftest_wait_timeout.restype = i32
    L.dspark_strerror.argtypes = [i32]
    L.dspark_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def _strerror(code):
    return _lib.dspark_strerror(int(code)).decode()


def library():
    """The loaded ctypes library (raises DSparkError if it is not built)."""
    return _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(code, where):
    if code != OK:
        raise DSparkError(code, where)


def _dt(t, what):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")


def _need(t, what, dtype=None, device=None):
    if t is None:
        raise ValueError(f"{what} is required")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return t


def _sized(t, what, shape):
    """Raise unless t has this shape.  The kernels index every tensor from the
    sizes alone, so a tensor smaller than its sizes say would be read or
    written past its end on the device."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    return t


_ws_cache = {}
_ws_views = {}


def workspace_size(B, gamma, V):
    return int(_load().dspark_workspace_size(B, gamma, V))


def workspace(B, gamma, V, device):
    """A cached, 256-byte aligned device workspace for these sizes."""
    view = _ws_views.get((B, gamma, V, device))
    if view is not None:
        return view
    n = workspace_size(B, gamma, V)
    key = (torch.device(device), n)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    off = (-ws.data_ptr()) % 256
    view = _ws_views[(B, gamma, V, device)] = ws[off:off + n]
    return view


def _round_dev(round_dev, dev):
    if round_dev is not None:
        _need(round_dev, "round_dev", torch.int64, dev)
        _sized(round_dev, "round_dev", (1,))
    return _ptr(round_dev)


def markov_draft(U, W1, W2, anchor, seed, rnd=0, ws=None, T_early=None, round_dev=None):
    """x [B,G] i32, p [B,G] f32, lse [B,G] f32 = the Markov draft of one round.
    T_early [B,G+1,V] f32: target logits whose rows j < G get their softmax
    statistics into ws while the draft runs (for verify(early_stats=True)).
    round_dev: int64 [1] device tensor holding the round index (rnd ignored)."""
    L = _load()
    _need(U, "U", torch.float32)
    dev = U.device
    B, G, V = U.shape
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev); _need(anchor, "anchor", torch.int32, dev)
    r = W1.shape[-1]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(anchor, "anchor", (B,))
    if T_early is not None:
        _need(T_early, "T_early", torch.float32, dev)
        _sized(T_early, "T_early", (B, G + 1, V))
    rd = _round_dev(round_dev, dev)
    x = torch.empty((B, G), dtype=torch.int32, device=dev)
    p = torch.empty((B, G), dtype=torch.float32, device=dev)
    lse = torch.empty((B, G), dtype=torch.float32, device=dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    _check(L.dspark_markov_draft_ex(_ptr(U), _ptr(T_early), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(anchor), B, G,
                                    V, r, seed, rnd, rd, _ptr(x), _ptr(p), _ptr(lse), _ptr(ws), ws.numel(),
                                    _stream(dev)), "markov_draft")
    return x, p, lse


def gated_markov_draft(U, W1, W2, gate_g, gate_c, anchor, seed, rnd=0, ws=None, T_early=None, round_dev=None):
    """x, p, lse of the draft with the gated recurrent head (s_k = e_k + a_k *
    s_{k-1}, a_k = sigmoid(gate_g * e_k + gate_c), e_k = W1[x_{k-1}]; bias
    s_k . W2).  gate_g, gate_c: float32 [r].  The states stay in ws for
    verify(gated=True).  Tensor-core path only (bf16, r = 256)."""
    L = _load()
    _need(U, "U", torch.float32)
    dev = U.device
    B, G, V = U.shape
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev); _need(anchor, "anchor", torch.int32, dev)
    r = W1.shape[-1]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(anchor, "anchor", (B,))
    _need(gate_g, "gate_g", torch.float32, dev); _need(gate_c, "gate_c", torch.float32, dev)
    _sized(gate_g, "gate_g", (r,)); _sized(gate_c, "gate_c", (r,))
    if T_early is not None:
        _need(T_early, "T_early", torch.float32, dev)
        _sized(T_early, "T_early", (B, G + 1, V))
    rd = _round_dev(round_dev, dev)
    x = torch.empty((B, G), dtype=torch.int32, device=dev)
    p = torch.empty((B, G), dtype=torch.float32, device=dev)
    lse = torch.empty((B, G), dtype=torch.float32, device=dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    _check(L.dspark_gated_markov_draft(_ptr(U), _ptr(T_early), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(gate_g),
                                       _ptr(gate_c), _ptr(anchor), B, G, V, r, seed, rnd, rd, _ptr(x), _ptr(p),
                                       _ptr(lse), _ptr(ws), ws.numel(), _stream(dev)), "gated_markov_draft")
    return x, p, lse


def confidence(h, W1, w, anchor, x, sts_T=None):
    """c [B,G] f32 = sigmoid(w . [h_k ; W1[x_{k-1}]] / T_k)."""
    L = _load()
    _need(h, "h")
    dev = h.device
    B, G, H = h.shape
    _need(W1, "W1", device=dev); _need(w, "w", torch.float32, dev)
    _need(anchor, "anchor", torch.int32, dev); _need(x, "x", torch.int32, dev)
    if sts_T is not None:
        _need(sts_T, "sts_T", torch.float32, dev)
    if W1.dim() != 2:
        raise ValueError(f"W1 must be [V, r], got {list(W1.shape)}")
    V, r = W1.shape
    _sized(w, "w", (H + r,)); _sized(anchor, "anchor", (B,)); _sized(x, "x", (B, G)); _sized(sts_T, "sts_T", (G,))
    c = torch.empty((B, G), dtype=torch.float32, device=dev)
    _check(L.dspark_confidence(_ptr(h), _dt(h, "h"), _ptr(W1), _dt(W1, "W1"), _ptr(w), _ptr(sts_T), _ptr(anchor),
                               _ptr(x), B, G, H, r, V, _ptr(c), _stream(dev)), "confidence")
    return c


def schedule(c, sps=None, mode=SCHED_GREEDY, rnd=0, khist=None, ws=None, round_dev=None):
    """ell [B] i32, nstar [1] i32, theta [1] f64 from confidences c [B,G]."""
    L = _load()
    _need(c, "c", torch.float32)
    dev = c.device
    B, G = c.shape
    if sps is not None:
        _need(sps, "sps", torch.float32, dev)
    if khist is not None:
        _need(khist, "khist", torch.int32, dev)
    _sized(khist, "khist", (2,))
    ell = torch.empty(B, dtype=torch.int32, device=dev)
    nstar = torch.empty(1, dtype=torch.int32, device=dev)
    theta = torch.empty(1, dtype=torch.float64, device=dev)
    ws = workspace(B, G, 8, dev) if ws is None else ws
    n_sps = 0 if sps is None else sps.numel()
    rd = _round_dev(round_dev, dev)
    _check(L.dspark_schedule_ex(_ptr(c), B, G, _ptr(sps), n_sps, mode, rnd, rd, _ptr(khist), _ptr(ell),
                                _ptr(nstar), _ptr(theta), _ptr(ws), ws.numel(), _stream(dev)), "schedule")
    return ell, nstar, theta


def verify(T, U, W1, W2, anchor, x, p_d, lse_d, ell, seed, rnd=0, ws=None, early_stats=False, round_dev=None,
           advance_round=False, scratch_from_draft=False, gated=False, all_row_stats=False):
    """n [B] i32 accepted counts, tok [B] i32 corrected / bonus tokens.
    early_stats: ws already holds the target-row statistics from
    markov_draft(T_early=T).  round_dev / advance_round: the round index as a
    device int64 [1], advanced by the call's last kernel.
    scratch_from_draft: a draft_schedule on ws cleared the call's scratch.
    gated: the draft was gated_markov_draft on ws (its states are the
    residual's bias operand).  all_row_stats: take the statistics of every
    row j < ell (for acceptance_label(stats="verify")) instead of only the
    rows the accept tests reach."""
    L = _load()
    _need(T, "T", torch.float32)
    dev = T.device
    _need(U, "U", torch.float32, dev)
    B, G, V = U.shape
    if tuple(T.shape) != (B, G + 1, V):
        raise ValueError(f"T must be [B, gamma+1, V] = {(B, G + 1, V)}, got {tuple(T.shape)}")
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev)
    for t, n in [(anchor, "anchor"), (x, "x"), (ell, "ell")]:
        _need(t, n, torch.int32, dev)
    _need(p_d, "p_d", torch.float32, dev); _need(lse_d, "lse_d", torch.float32, dev)
    r = W1.shape[-1]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(anchor, "anchor", (B,)); _sized(ell, "ell", (B,))
    for t, n in [(x, "x"), (p_d, "p_d"), (lse_d, "lse_d")]:
        _sized(t, n, (B, G))
    n = torch.empty(B, dtype=torch.int32, device=dev)
    tok = torch.empty(B, dtype=torch.int32, device=dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    rd = _round_dev(round_dev, dev)
    flags = ((EARLY_TARGET_STATS if early_stats else 0) | (ADVANCE_ROUND if advance_round else 0) |
             (SCRATCH_FROM_DRAFT if scratch_from_draft else 0) | (GATED_STATES if gated else 0) |
             (ALL_ROW_STATS if all_row_stats else 0))
    _check(L.dspark_verify_ex(_ptr(T), _ptr(U), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(anchor), _ptr(x),
                              _ptr(p_d), _ptr(lse_d), _ptr(ell), B, G, V, r, seed, rnd, rd, flags, _ptr(n), _ptr(tok),
                              _ptr(ws), ws.numel(), _stream(dev)), "verify")
    return n, tok


def acceptance_label(T, U, W1, W2, anchor, x, lse_d, ell, ws=None, stats=None):
    """label [B, gamma] f32: sum_v min(p_d, p_t) for every verified position
    k <= ell[b] (0 elsewhere).  Tensor-core path only (bf16, r = 256).
    stats: None (the call streams the target rows' statistics first),
    "early" (ws holds them from markov_draft(T_early=T)) or "verify" (ws
    holds them from a verify or round with all_row_stats=True)."""
    L = _load()
    _need(T, "T", torch.float32)
    dev = T.device
    _need(U, "U", torch.float32, dev)
    B, G, V = U.shape
    if tuple(T.shape) != (B, G + 1, V):
        raise ValueError(f"T must be [B, gamma+1, V] = {(B, G + 1, V)}, got {tuple(T.shape)}")
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev)
    for t, n in [(anchor, "anchor"), (x, "x"), (ell, "ell")]:
        _need(t, n, torch.int32, dev)
    _need(lse_d, "lse_d", torch.float32, dev)
    r = W1.shape[-1]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(anchor, "anchor", (B,)); _sized(ell, "ell", (B,))
    _sized(x, "x", (B, G)); _sized(lse_d, "lse_d", (B, G))
    label = torch.empty(B, G, dtype=torch.float32, device=dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    flags = {None: 0, "early": EARLY_TARGET_STATS, "verify": TARGET_STATS_FROM_VERIFY}[stats]
    _check(L.dspark_acceptance_label_ex(_ptr(T), _ptr(U), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(anchor), _ptr(x),
                                        _ptr(lse_d), _ptr(ell), B, G, V, r, flags, _ptr(label), _ptr(ws), ws.numel(),
                                        _stream(dev)), "acceptance_label")
    return label


def sts_fit(z, ell, acc, grid):
    """Sequential temperature scaling: (T [gamma] f32, ece [gamma] f32) fitted on
    the samples (z [N, gamma] f32 logits, ell and acc [N] i32) over the grid of
    temperatures (f32), all on one device."""
    L = _load()
    _need(z, "z", torch.float32)
    dev = z.device
    N, G = z.shape
    _need(ell, "ell", torch.int32, dev); _need(acc, "acc", torch.int32, dev); _need(grid, "grid", torch.float32, dev)
    _sized(ell, "ell", (N,)); _sized(acc, "acc", (N,)); _sized(grid, "grid", (grid.numel(),))
    T = torch.empty(G, dtype=torch.float32, device=dev)
    e = torch.empty(G, dtype=torch.float32, device=dev)
    nbytes = L.dspark_sts_workspace_size(N, G, grid.numel())
    ws = torch.empty(max(256, nbytes), dtype=torch.uint8, device=dev)
    _check(L.dspark_sts_fit(_ptr(z), _ptr(ell), _ptr(acc), N, G, _ptr(grid), grid.numel(), _ptr(T), _ptr(e), _ptr(ws),
                            ws.numel(), _stream(dev)), "sts_fit")
    return T, e


_INT_MAX = 2 ** 31 - 1   # of the library's sizes; a larger one would wrap around on its way there
_ROW_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _address(t):
    return None if t is None else t.data_ptr()


def _launch(fn, where, dev, *args):
    """fn(*args, stream) on the current stream of dev, with dev current (the
    library launches on the current device).  These calls take ten
    microseconds on the GPU for a few rows, so the host's share is kept small:
    plain addresses, and the stream's handle without a stream object."""
    if torch.cuda.current_device() == dev.index:
        code = fn(*args, _stream_handle(dev.index))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _stream_handle(dev.index))
    if code != OK:
        raise DSparkError(code, where)


# (a private name of torch, with the public way where a version lacks it)
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _row_args(logits, rows, what="logits"):
    """device, leading shape, N, R, V, row stride and dtype code of rows of logits."""
    if logits is None or not logits.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if logits.dtype not in _ROW_DTYPES:
        raise TypeError(f"{what} must be float32, bfloat16 or float16, got {logits.dtype}")
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError(f"{what} must be [..., V] with V >= 1, got {list(logits.shape)}")
    lead, V = tuple(logits.shape[:-1]), logits.shape[-1]
    N = math.prod(lead)
    if max(N, V) > _INT_MAX:
        raise DSparkError(ERR_UNSUPPORTED, f"{what} of {list(logits.shape)}")
    if V > 1 and N > 0 and logits.stride(-1) != 1:
        raise ValueError(f"{what} must have entries of a row next to each other")
    stride = V
    if N > 1 and not logits.is_contiguous():
        try:
            stride = logits.view(N, V).stride(0)
        except RuntimeError:
            raise ValueError(f"{what} must have rows a fixed distance apart (strides {logits.stride()})") from None
        if stride < V:
            raise ValueError(f"{what} must not have overlapping rows (strides {logits.stride()})")
    R = 1
    if rows is not None:
        if len(lead) != 2:
            raise ValueError(f"rows needs {what} [B, R, V], got {list(logits.shape)}")
        _need(rows, "rows", torch.int32, logits.device)
        _sized(rows, "rows", lead[:1])
        R = max(lead[1], 1)
    return logits.device, lead, N, R, V, stride, _ROW_DTYPES[logits.dtype]


def _row_vector(t, what, lead, dev, dtype=torch.float32):
    if t is not None:
        _need(t, what, dtype, dev)
        _sized(t, what, lead)
    return _ptr(t)


def _gradient_out(out, logits, dtype):
    """A dense gradient of these logits, checked or allocated.  It may be the
    logits themselves, and may not overlap them in another way."""
    if out is None:
        return torch.empty(logits.shape, dtype=dtype, device=logits.device)
    _need(out, "out", dtype, logits.device)
    _sized(out, "out", logits.shape)
    if out.numel() > 0:
        a0, b0 = out.data_ptr(), logits.data_ptr()
        last = sum((n - 1) * s for n, s in zip(logits.shape, logits.stride()))
        a1, b1 = a0 + out.numel() * out.element_size(), b0 + (last + 1) * logits.element_size()
        same = a0 == b0 and logits.dtype == dtype and logits.is_contiguous()
        if a0 < b1 and b0 < a1 and not same:
            raise ValueError("out overlaps the logits; it may only be the same dense tensor")
    return out


def _logprob_outputs(lead, top_k, dev):
    logp, entropy, lse = (torch.empty(lead, dtype=torch.float32, device=dev) for _ in range(3))
    if not top_k:
        return logp, entropy, lse, None, None
    return (logp, entropy, lse, torch.empty((*lead, top_k), dtype=torch.int32, device=dev),
            torch.empty((*lead, top_k), dtype=torch.float32, device=dev))


def token_logprobs(logits, tokens, top_k=0, rows=None):
    """logp, entropy, lse [...] f32 of logits [..., V] (f32, bf16 or f16, rows a
    fixed distance apart) at tokens [...] i32 (-1: none), and the top_k <= 128
    most probable entries of each row, largest first and equal ones by index:
    top_idx i32, top_logp f32 [..., top_k] (None with top_k = 0).
    rows [B] i32, with logits [B, R, V]: only the first rows[b] rows of b count
    (the others' outputs are 0, -1 and -inf)."""
    L = _load()
    dev, lead, N, R, V, stride, dt = _row_args(logits, rows)
    _row_vector(_need(tokens, "tokens"), "tokens", lead, dev, torch.int32)
    out = _logprob_outputs(lead, _top_k(top_k, V), dev)
    _launch(L.dspark_token_logprobs, "token_logprobs", dev, logits.data_ptr(), dt, stride, tokens.data_ptr(),
            _address(rows), N, R, V, top_k, *map(_address, out))
    return out


def _top_k(top_k, V):
    if not 0 <= top_k <= V:
        raise ValueError(f"top_k must be in [0, V = {V}], got {top_k}")
    return top_k


def emitted_logprobs(T, x, n, tok, top_k=0):
    """token_logprobs of the tokens a round emitted, from its target logits T
    [B, G+1, V] and its outputs x [B, G], n and tok [B]: row j < n[b] scores
    x[b, j], row n[b] scores tok[b], and the rows after it do not count."""
    L = _load()
    dev, lead, N, _, V, stride, dt = _row_args(T, None, "T")
    if len(lead) != 2 or lead[1] < 2 or not T.is_contiguous():
        raise ValueError(f"T must be [B, gamma+1, V] and contiguous, got {list(T.shape)}")
    B, G = lead[0], lead[1] - 1
    for t, name, shape in [(x, "x", (B, G)), (n, "n", (B,)), (tok, "tok", (B,))]:
        _row_vector(_need(t, name), name, shape, dev, torch.int32)
    out = _logprob_outputs(lead, _top_k(top_k, V), dev)
    _launch(L.dspark_emitted_logprobs, "emitted_logprobs", dev, T.data_ptr(), dt, x.data_ptr(), n.data_ptr(),
            tok.data_ptr(), B, G, V, top_k, *map(_address, out))
    return out


def token_logprobs_backward(logits, tokens, lse, entropy=None, g_logp=None, g_entropy=None, rows=None, out=None):
    """The gradient of the logits, of their type and dense, from the upstream
    gradients g_logp and g_entropy [...] f32 (None: 0) of token_logprobs' logp
    and entropy; lse and entropy are that call's outputs.  out: a dense tensor
    to write, which may be the logits themselves."""
    L = _load()
    dev, lead, N, R, V, stride, dt = _row_args(logits, rows)
    _row_vector(_need(tokens, "tokens"), "tokens", lead, dev, torch.int32)
    _row_vector(_need(lse, "lse"), "lse", lead, dev)
    if g_entropy is not None:
        _need(entropy, "entropy")
    for t, name in [(entropy, "entropy"), (g_logp, "g_logp"), (g_entropy, "g_entropy")]:
        _row_vector(t, name, lead, dev)
    out = _gradient_out(out, logits, logits.dtype)
    _launch(L.dspark_token_logprobs_backward, "token_logprobs_backward", dev, logits.data_ptr(), dt, stride,
            tokens.data_ptr(), lse.data_ptr(), _address(entropy), _address(g_logp), _address(g_entropy),
            _address(rows), N, R, V, out.data_ptr())
    return out


def _distill_args(logits, top_idx, top_val, teacher_lse, rows, temperature):
    dev, lead, N, R, V, stride, dt = _row_args(logits, rows)
    _need(top_idx, "top_idx", torch.int32, dev); _need(top_val, "top_val", torch.float32, dev)
    if top_idx.dim() != len(lead) + 1 or top_idx.shape[-1] < 1:
        raise ValueError(f"top_idx must be {list(lead)} + [K], got {list(top_idx.shape)}")
    K = top_idx.shape[-1]
    if K > _INT_MAX:
        raise DSparkError(ERR_UNSUPPORTED, f"top_idx of {list(top_idx.shape)}")
    _sized(top_idx, "top_idx", (*lead, K)); _sized(top_val, "top_val", (*lead, K))
    _row_vector(teacher_lse, "teacher_lse", lead, dev)
    if not 0.0 < temperature < math.inf:
        raise ValueError(f"temperature must be positive and finite, got {temperature}")
    return dev, lead, N, R, V, stride, dt, K


def distill_loss(logits, top_idx, top_val, temperature=1.0, teacher_lse=None, weight=None, rows=None, grad=False,
                 grad_dtype=None, out=None):
    """Kullback-Leibler loss of a student's logits [..., V] against a teacher's K
    kept logits top_val [..., K] f32 at top_idx [..., K] i32 (-1: absent; K <= 128):
    loss [...] f32, stats [..., 2] f32 (for distill_loss_backward) and, with
    grad, weight * d loss / d logits of type grad_dtype (the logits' own, or
    bfloat16 for float32 logits), else None, in one call.
    teacher_lse [...] f32, the log-sum-exp of the teacher's whole row of
    top_val / temperature: the teacher's remaining mass is matched, as one
    bucket, with the student's; None: the kept entries are renormalised.
    weight [...] f32 (None: 1) scales the gradient, not the loss.
    rows as in token_logprobs; out as in token_logprobs_backward."""
    L = _load()
    dev, lead, N, R, V, stride, dt, K = _distill_args(logits, top_idx, top_val, teacher_lse, rows, temperature)
    _row_vector(weight, "weight", lead, dev)
    if not grad and (out is not None or grad_dtype is not None):
        raise ValueError("out and grad_dtype need grad")
    gdt = logits.dtype if grad_dtype is None else grad_dtype
    if gdt not in _ROW_DTYPES:
        raise TypeError(f"grad_dtype must be float32, bfloat16 or float16, got {gdt}")
    dlogits = _gradient_out(out, logits, gdt) if grad else None
    loss = torch.empty(lead, dtype=torch.float32, device=dev)
    stats = torch.empty((*lead, 2), dtype=torch.float32, device=dev)
    _launch(L.dspark_distill_loss, "distill_loss", dev, logits.data_ptr(), dt, stride, top_idx.data_ptr(),
            top_val.data_ptr(), _address(teacher_lse), _address(weight), _address(rows), N, R, V, K, temperature,
            loss.data_ptr(), stats.data_ptr(), _address(dlogits), _ROW_DTYPES[gdt])
    return loss, stats, dlogits


def distill_loss_backward(logits, top_idx, top_val, stats, g, temperature=1.0, teacher_lse=None, rows=None,
                          grad_dtype=None, out=None):
    """g * d loss / d logits of distill_loss from its stats and an upstream
    gradient g [...] f32; the other arguments as for that call."""
    L = _load()
    dev, lead, N, R, V, stride, dt, K = _distill_args(logits, top_idx, top_val, teacher_lse, rows, temperature)
    _row_vector(_need(stats, "stats"), "stats", (*lead, 2), dev)
    _row_vector(_need(g, "g"), "g", lead, dev)
    gdt = logits.dtype if grad_dtype is None else grad_dtype
    if gdt not in _ROW_DTYPES:
        raise TypeError(f"grad_dtype must be float32, bfloat16 or float16, got {gdt}")
    out = _gradient_out(out, logits, gdt)
    _launch(L.dspark_distill_loss_backward, "distill_loss_backward", dev, logits.data_ptr(), dt, stride,
            top_idx.data_ptr(), top_val.data_ptr(), stats.data_ptr(), g.data_ptr(), _address(teacher_lse),
            _address(rows), N, R, V, K, temperature, out.data_ptr(), _ROW_DTYPES[gdt])
    return out


def _head_args(logits, what, dtype, W1, W2, anchor, x):
    _need(logits, what, dtype)
    dev = logits.device
    if logits.dim() != 3:
        raise ValueError(f"{what} must be [B, gamma, V], got {list(logits.shape)}")
    B, G, V = logits.shape
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev)
    _need(anchor, "anchor", torch.int32, dev); _need(x, "x", torch.int32, dev)
    r = W1.shape[-1]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(anchor, "anchor", (B,)); _sized(x, "x", (B, G))
    return dev, B, G, V, r


_head_status = {}


def head_status(device):
    """The status word of the calls of markov_logits, markov_head_backward,
    linear_cross_entropy(_backward) and newton_schulz on this device that were given
    no ws, for read_status.  (A call that is captured into a graph before the device
    has one takes a word of its own, which nobody reads: call this first, or give it
    a ws.)"""
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    st = _head_status.get(dev)
    if st is None:
        st = torch.zeros(256, dtype=torch.uint8, device=dev)
        # (cleared before another stream's call can record in it)
        torch.cuda.current_stream(dev).synchronize()
        st = _head_status.setdefault(dev, st)   # (the one that another thread made meanwhile)
    return st


def _status_without_ws(dev):
    st = _head_status.get(dev)
    if st is None:
        with torch.cuda.device(dev):
            capturing = torch.cuda.is_current_stream_capturing()
        st = torch.zeros(256, dtype=torch.uint8, device=dev) if capturing else head_status(dev)
    return st


def markov_logits(U, W1, W2, anchor, x, dtype=torch.float32, ws=None, out=None):
    """l [B, G, V] = U + W1[x_{k-1}] W2^T (x_0 = anchor), the logits the draft
    samples from at tokens x [B, G], as float32 or bfloat16.  out: a tensor to
    write, which may be U itself (float32).  Tensor-core path only (bf16
    weights, r = 256).  ws: 256 zeroed bytes to read_status of; by default
    errors are recorded in head_status."""
    L = _load()
    dev, B, G, V, r = _head_args(U, "U", torch.float32, W1, W2, anchor, x)
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    out = _gradient_out(out, U, dtype)
    ws = _status_without_ws(dev) if ws is None else _need(ws, "ws", torch.uint8, dev)
    _launch(L.dspark_markov_logits, "markov_logits", dev, U.data_ptr(), W1.data_ptr(), W2.data_ptr(), _dt(W1, "W1"),
            anchor.data_ptr(), x.data_ptr(), B, G, V, r, out.data_ptr(), _ROW_DTYPES[dtype], ws.data_ptr(), ws.numel())
    return out


def head_workspace(B, gamma, V, device):
    """A workspace of markov_head_backward for these sizes."""
    ws = _head_workspace(B, gamma, V, device)
    ws[:256].zero_()
    return ws


def _head_workspace(B, gamma, V, device):
    n = int(_load().dspark_head_workspace_size(B, gamma, V))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def markov_head_backward(dlogits, W1, W2, anchor, x, ws=None):
    """dW1, dW2 [V, r] f32 from the gradient dlogits [B, G, V] bf16 of
    markov_logits.  ws: a head_workspace to keep (and read_status of); by
    default one is allocated for the call and errors are recorded in head_status."""
    L = _load()
    dev, B, G, V, r = _head_args(dlogits, "dlogits", torch.bfloat16, W1, W2, anchor, x)
    dW1 = torch.empty((V, r), dtype=torch.float32, device=dev)
    dW2 = torch.empty((V, r), dtype=torch.float32, device=dev)
    status = None
    if ws is None:
        ws, status = _head_workspace(B, G, V, dev), _status_without_ws(dev)
    else:
        _need(ws, "ws", torch.uint8, dev)
    _launch(L.dspark_markov_head_backward_ex, "markov_head_backward", dev, dlogits.data_ptr(), W1.data_ptr(),
            W2.data_ptr(), _dt(W1, "W1"), anchor.data_ptr(), x.data_ptr(), B, G, V, r, _address(status), dW1.data_ptr(),
            dW2.data_ptr(), ws.data_ptr(), ws.numel())
    return dW1, dW2


def _hidden_args(h, W, tokens, rows):
    """device, leading shape, N, R, V, D, both row strides and the dtype code of
    hidden states and the head over them."""
    dev, lead, N, R, D, h_stride, dt = _row_args(h, rows, "h")
    if W is None or not W.is_cuda:
        raise ValueError("W must be a CUDA tensor")
    if W.device != dev:
        raise ValueError(f"W is on {W.device}, expected {dev}")
    if W.dtype != h.dtype:
        raise TypeError(f"W must be {h.dtype}, got {W.dtype}")
    if W.dim() != 2 or W.shape[0] < 1 or W.shape[1] != D:
        raise ValueError(f"W must be [V, {D}] with V >= 1, got {list(W.shape)}")
    V, (W_stride, step) = W.shape[0], W.stride()
    if V > _INT_MAX:
        raise DSparkError(ERR_UNSUPPORTED, f"W of {list(W.shape)}")
    if D > 1 and step != 1:
        raise ValueError("W must have entries of a row next to each other")
    if V == 1:
        W_stride = D
    elif W_stride < D:
        raise ValueError(f"W must not have overlapping rows (strides {W.stride()})")
    _row_vector(_need(tokens, "tokens"), "tokens", lead, dev, torch.int32)
    return dev, lead, N, R, V, D, h_stride, W_stride, dt


@functools.lru_cache(maxsize=1024)
def _hidden_workspace_size(N, V, D, what):
    return max(int(_load().dspark_linear_ce_workspace_size(N, V, D, what)), 256)


def _hidden_workspace(ws, N, V, D, what, dev):
    """A workspace, and the word that errors are recorded in when it is not the caller's."""
    if ws is not None:
        return _need(ws, "ws", torch.uint8, dev), None
    return torch.empty(_hidden_workspace_size(N, V, D, what), dtype=torch.uint8, device=dev), _status_without_ws(dev)


def linear_ce_workspace(N, V, D, device, dh=False, dW=False):
    """A workspace of linear_cross_entropy for N rows (dh and dW False), or of
    linear_cross_entropy_backward for these gradients."""
    n = _hidden_workspace_size(N, V, D, int(bool(dh)) + 2 * int(bool(dW)))
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def linear_cross_entropy(h, W, tokens, rows=None, ws=None):
    """loss, lse [...] f32: the softmax cross entropy of tokens [...] i32 (-1:
    none) under the logits h W^T of hidden states h [..., D] and a head W [V, D]
    (bfloat16 or float16; rows a fixed distance apart, W's on 16 bytes; D % 8 ==
    0), which are formed in pieces of the vocabulary and not kept.
    rows [B] i32, with h [B, R, D]: only the first rows[b] rows of b count.  Rows
    that do not count, or have no token, cost next to nothing and give zeros.
    ws: a linear_ce_workspace to keep (and read_status of); by default one is
    allocated for the call and errors are recorded in head_status."""
    L = _load()
    dev, lead, N, R, V, D, h_stride, W_stride, dt = _hidden_args(h, W, tokens, rows)
    loss = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev)
    ws, status = _hidden_workspace(ws, N, V, D, 0, dev)
    _launch(L.dspark_linear_cross_entropy, "linear_cross_entropy", dev, h.data_ptr(), h_stride, W.data_ptr(), W_stride, dt,
            tokens.data_ptr(), _address(rows), N, R, V, D, loss.data_ptr(), lse.data_ptr(), _address(status),
            ws.data_ptr(), ws.numel())
    return loss, lse


def linear_cross_entropy_backward(h, W, tokens, lse, g_loss, g_lse=None, rows=None, dh=True, dW=True, ws=None):
    """dh [..., D] and dW [V, D], of h's type (None where dh or dW is False), from
    the lse of linear_cross_entropy and the upstream gradients g_loss and g_lse
    [...] f32 (None: 0); the other arguments as for that call.  Slopes are rounded to
    h's type on the way; with more than 128 rows that count a bf16 dW is off by
    2.2e-3 of its 2-norm, where its own rounding takes 1.7e-3."""
    L = _load()
    dev, lead, N, R, V, D, h_stride, W_stride, dt = _hidden_args(h, W, tokens, rows)
    _row_vector(_need(lse, "lse"), "lse", lead, dev)
    _row_vector(_need(g_loss, "g_loss"), "g_loss", lead, dev)
    _row_vector(g_lse, "g_lse", lead, dev)
    if not dh and not dW:
        raise ValueError("one of dh and dW is needed")
    ws, status = _hidden_workspace(ws, N, V, D, int(bool(dh)) + 2 * int(bool(dW)), dev)
    dh = torch.empty(h.shape, dtype=h.dtype, device=dev) if dh else None
    dW = torch.empty((V, D), dtype=W.dtype, device=dev) if dW else None
    _launch(L.dspark_linear_cross_entropy_backward, "linear_cross_entropy_backward", dev, h.data_ptr(), h_stride,
            W.data_ptr(), W_stride, dt, tokens.data_ptr(), _address(rows), lse.data_ptr(), g_loss.data_ptr(),
            _address(g_lse), N, R, V, D, _address(dh), _address(dW), _address(status), ws.data_ptr(), ws.numel())
    return dh, dW


def newton_schulz_workspace(rows, cols, device):
    """A workspace of newton_schulz for an update of these sizes."""
    n = int(_load().dspark_newton_schulz_workspace_size(rows, cols))
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def newton_schulz(update, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, ws=None):
    """The update [rows, cols] (f32, bf16 or f16, rows a fixed distance apart)
    orthogonalised: X = update / (its Frobenius norm + eps), then `steps` times
    X <- a X + (b A + c A A) X with A = X X^T and (a, b, c) = coefficients; bfloat16.
    The default coefficients, Muon's, bring the singular values to between 0.7 and
    1.2 or so in five steps.  ws: a newton_schulz_workspace to keep (and
    read_status of); by default one is allocated for the call and errors are
    recorded in head_status."""
    L = _load()
    if update is not None and update.dim() != 2:
        raise ValueError(f"update must be [rows, cols], got {list(update.shape)}")
    if update is not None and update.is_cuda and update.numel() == 0:
        return torch.empty(update.shape, dtype=torch.bfloat16, device=update.device)
    dev, _, rows, _, cols, stride, dt = _row_args(update, None, "update")
    a, b, c = coefficients
    if not all(map(math.isfinite, (a, b, c, eps))) or eps < 0:
        raise ValueError(f"coefficients and eps >= 0 must be finite, got {coefficients} and {eps}")
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    status = None
    if ws is None:
        n = int(L.dspark_newton_schulz_workspace_size(rows, cols))
        ws, status = torch.empty(max(n, 256), dtype=torch.uint8, device=dev), _status_without_ws(dev)
    else:
        _need(ws, "ws", torch.uint8, dev)
    _launch(L.dspark_newton_schulz, "newton_schulz", dev, update.data_ptr(), dt, stride, rows, cols, steps, a, b, c, eps,
            out.data_ptr(), _address(status), ws.data_ptr(), ws.numel())
    return out


class RoundOutputs:
    """Device output buffers of one round (reused across rounds)."""

    def __init__(self, B, G, device):
        i32, f32 = torch.int32, torch.float32
        self.x = torch.empty((B, G), dtype=i32, device=device)
        self.p = torch.empty((B, G), dtype=f32, device=device)
        self.lse = torch.empty((B, G), dtype=f32, device=device)
        self.c = torch.empty((B, G), dtype=f32, device=device)
        self.ell = torch.empty(B, dtype=i32, device=device)
        self.nstar = torch.empty(1, dtype=i32, device=device)
        self.theta = torch.empty(1, dtype=torch.float64, device=device)
        self.n = torch.empty(B, dtype=i32, device=device)
        self.tok = torch.empty(B, dtype=i32, device=device)

    def as_dict(self):
        return dict(x=self.x, p=self.p, lse=self.lse, c=self.c, ell=self.ell, nstar=self.nstar,
                    theta=self.theta, n=self.n, tok=self.tok)

    def check(self, B, G, device):
        """Raise unless every buffer has the shape, dtype and device of a
        round of B requests and G positions."""
        i32, f32 = torch.int32, torch.float32
        want = dict(x=((B, G), i32), p=((B, G), f32), lse=((B, G), f32), c=((B, G), f32), ell=((B,), i32),
                    nstar=((1,), i32), theta=((1,), torch.float64), n=((B,), i32), tok=((B,), i32))
        for name, (shape, dtype) in want.items():
            t = getattr(self, name)
            _need(t, f"out.{name}", dtype, device)
            _sized(t, f"out.{name}", shape)


def _round_args(U, T, W1, W2, h, w, anchor, sps, khist, sts_T):
    # shared checks of round and draft_schedule (T may be None for the latter)
    _need(U, "U", torch.float32)
    dev = U.device
    B, G, V = U.shape
    if T is not None:
        _need(T, "T", torch.float32, dev)
        if tuple(T.shape) != (B, G + 1, V):
            raise ValueError(f"T must be [B, gamma+1, V] = {(B, G + 1, V)}, got {tuple(T.shape)}")
    _need(W1, "W1", device=dev); _need(W2, "W2", W1.dtype, dev); _need(h, "h", device=dev)
    _need(w, "w", torch.float32, dev); _need(anchor, "anchor", torch.int32, dev)
    if sps is not None:
        _need(sps, "sps", torch.float32, dev)
    if khist is not None:
        _need(khist, "khist", torch.int32, dev)
    if sts_T is not None:
        _need(sts_T, "sts_T", torch.float32, dev)
    if h.dim() != 3:
        raise ValueError(f"h must be [B, gamma, H], got {list(h.shape)}")
    r, H = W1.shape[-1], h.shape[2]
    _sized(W1, "W1", (V, r)); _sized(W2, "W2", (V, r)); _sized(h, "h", (B, G, H)); _sized(w, "w", (H + r,))
    _sized(anchor, "anchor", (B,)); _sized(khist, "khist", (2,)); _sized(sts_T, "sts_T", (G,))
    return dev, B, G, V, r, H


def draft_schedule(U, W1, W2, h, w, anchor, seed, rnd=0, sps=None, mode=SCHED_GREEDY, khist=None, sts_T=None,
                   out=None, ws=None, T_early=None, round_dev=None, chain_stats=False):
    """The first stage of a round (draft, confidence head, schedule; one
    persistent launch on the tensor-core path) into out.x, p, lse, c, ell,
    nstar, theta.  T_early: target logits whose statistics the draft takes
    along (chain_stats: only of the rows the accept tests can reach; verify
    with early_stats=True either way).  Returns the RoundOutputs."""
    L = _load()
    if chain_stats and T_early is None:
        raise ValueError("chain_stats needs T_early")
    dev, B, G, V, r, H = _round_args(U, T_early, W1, W2, h, w, anchor, sps, khist, sts_T)
    out = RoundOutputs(B, G, dev) if out is None else out
    out.check(B, G, dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    n_sps = 0 if sps is None else sps.numel()
    rd = _round_dev(round_dev, dev)
    _check(L.dspark_draft_schedule_ex(_ptr(U), _ptr(T_early), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(h),
                                      _dt(h, "h"), _ptr(w), _ptr(sts_T), _ptr(anchor), B, G, V, r, H, _ptr(sps),
                                      n_sps, mode, _ptr(khist), seed, rnd, rd,
                                      CHAIN_TARGET_STATS if chain_stats else 0, _ptr(out.x), _ptr(out.p),
                                      _ptr(out.lse), _ptr(out.c), _ptr(out.ell), _ptr(out.nstar), _ptr(out.theta),
                                      _ptr(ws), ws.numel(), _stream(dev)), "draft_schedule")
    return out


def round(U, T, W1, W2, h, w, anchor, seed, rnd=0, sps=None, mode=SCHED_GREEDY, khist=None, sts_T=None,
          out=None, ws=None, early_stats=False, round_dev=None, advance_round=False, all_row_stats=False,
          chain_stats=False):
    """One whole round (draft, confidence, schedule, verify) on U's device.
    early_stats: the draft takes the target rows' statistics while it runs.
    chain_stats: the draft takes those of the rows the accept tests reach.
    all_row_stats: verification takes the statistics of every row j < ell
    (otherwise only the rows the accept tests reach).
    round_dev / advance_round: the round index as a device int64 [1] (rnd
    ignored), advanced by the round's last kernel.
    Returns a RoundOutputs (device tensors)."""
    L = _load()
    _need(T, "T", torch.float32)
    dev, B, G, V, r, H = _round_args(U, T, W1, W2, h, w, anchor, sps, khist, sts_T)
    out = RoundOutputs(B, G, dev) if out is None else out
    out.check(B, G, dev)
    ws = workspace(B, G, V, dev) if ws is None else ws
    n_sps = 0 if sps is None else sps.numel()
    rd = _round_dev(round_dev, dev)
    flags = ((EARLY_TARGET_STATS if early_stats else 0) | (ADVANCE_ROUND if advance_round else 0) |
             (ALL_ROW_STATS if all_row_stats else 0) | (CHAIN_TARGET_STATS if chain_stats else 0))
    _check(L.dspark_round_ex(_ptr(U), _ptr(T), _ptr(W1), _ptr(W2), _dt(W1, "W1"), _ptr(h), _dt(h, "h"), _ptr(w),
                             _ptr(sts_T), _ptr(anchor), B, G, V, r, H, _ptr(sps), n_sps, mode, _ptr(khist), seed,
                             rnd, rd, flags, _ptr(out.x), _ptr(out.p), _ptr(out.lse), _ptr(out.c), _ptr(out.ell),
                             _ptr(out.nstar), _ptr(out.theta), _ptr(out.n), _ptr(out.tok), _ptr(ws), ws.numel(),
                             _stream(dev)), "round")
    return out


def selftest_wait_timeout(mode, ws):
    """Enqueue the bounded-wait self-test (mode 0: mbarrier, 1: grid barrier);
    its status word then reads ERR_TIMEOUT (see read_status)."""
    L = _load()
    _check(L.dspark_selftest_wait_timeout(int(mode), _ptr(ws), ws.numel(), _stream(ws.device)),
           "selftest_wait_timeout")


def read_status(ws, device=None):
    """Synchronise the current stream and return (and clear) the status word."""
    L = _load()
    st = ctypes.c_int(0)
    dev = ws.device if device is None else device
    _check(L.dspark_read_status(_ptr(ws), ctypes.byref(st), _stream(dev)), "read_status")
    return int(st.value)
