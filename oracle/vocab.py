"""Losses over a vocabulary and their gradients in 64 bits (oracle), with how far a call may be off.

Written with torch in float64, so that a test can put large cases on whatever device it likes; only elementary
operations and products of two matrices. Rows that are left out, and entries that are not there, are taken out before
anything is computed of them.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24      # the largest relative error of a rounding to fp32
U_BF16 = 2.0 ** -8  # and to bf16


def teacher(logits, ids, temperature):
    """(q, log q) over a row's entries: 0 where there is none; rows without entries are all 0."""
    there = ids >= 0
    x = torch.where(there, logits.double(), torch.full_like(logits, -math.inf, dtype=torch.float64)) / temperature
    top = x.max(1, keepdim=True)[0]
    empty = top == -math.inf
    e = torch.where(there, torch.exp(x - torch.where(empty, torch.zeros_like(top), top)), torch.zeros_like(x))
    total = torch.where(empty, torch.ones_like(top), e.sum(1, keepdim=True))
    q = e / total
    log_q = torch.where(q != 0, x - torch.where(empty, torch.zeros_like(top), top) - torch.log(total), torch.zeros_like(x))
    return torch.where(empty, torch.zeros_like(q), q), log_q


def loss_and_gradients(hidden, weight, ids, logits=None, reduction="mean", temperature=1.0, token_weights=None,
                       ignore_index=-100, dtype=None, d_terms=1):
    """(loss, d_hidden, d_weight), and with dtype ("fp32" or "bf16", what a call computes in) their bounds behind them.
    d_terms: of how many bf16 values, each the rounding of what the ones before leave, a bf16 call's D is the sum.

    The bounds, all in absolute terms, with A = |h| |W|^T / temperature:
    * logits: H products and sums in fp32, and a rounding of the scale: (H + 8) U A; fp32 operands are three bf16
      terms, six products of which are summed (6 H sums, and 2 U A for those left out): (6 H + 16) U A;
    * statistics: a shift of all logits by at most dz changes log-sum-exp by at most that; exponentials are off by 4 U
      and what rounds their argument, U (|z| + |lse|) log2(e), sums by U for each of at most 192 levels;
    * losses: both, the target's own logit, and a rounding of every operation (16 U of every term);
    * D = c (p - q): p's relative error is that of its exponent; in bf16 D is rounded, U_BF16 to the power of d_terms, and exp(z - m) to fp16
      times 2^14, 2^-11 of it or, below the smallest normal value, 2^-25, which is 2^-39 of the largest; in fp32 a
      few U;
    * products of D: its error times the other operand, a sum of fp32 terms in any order (n U of the terms'
      magnitudes), the rounding of the result;
    * values below the smallest normal one, 2^-126, may be lost: the exponential (then times c), D itself, the terms
      of its products, the result.
    """
    T, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    K = 1 if logits is None else logits.shape[1]
    ids2 = ids.reshape(T, K).long()
    if logits is None:
        out = ids2[:, 0] == ignore_index
        bad = ~out & ((ids2[:, 0] < 0) | (ids2[:, 0] >= V))
        q = torch.ones(T, 1, dtype=torch.float64, device=dev)
        log_q = torch.zeros_like(q)
    else:
        bad = (ids2 >= V).any(1)
        q, log_q = teacher(logits, ids2, temperature)
        there = ids2 >= 0
        out = ~bad & ~((there & (logits != -math.inf)).any(1))
    w = torch.ones(T, dtype=torch.float64, device=dev) if token_weights is None else token_weights.double()
    take = (~out & ~bad & (w != 0)).nonzero()[:, 0]
    count = int((~out).sum())
    h, W = hidden[take].double(), weight.double()
    own = ids2[take]
    q, log_q, w = q[take], log_q[take], w[take]
    there = own >= 0
    at = torch.where(there, own, torch.zeros_like(own))
    q = torch.where(there, q, torch.zeros_like(q))
    z = h @ W.t() / temperature
    top = z.max(1, keepdim=True)[0] if len(take) else z.new_zeros(0, 1)
    e = torch.exp(z - top)
    lse = top + torch.log(e.sum(1, keepdim=True))
    p = torch.exp(z - lse)
    zt = z.gather(1, at)
    terms = torch.where(q != 0, q * (log_q + lse - zt), torch.zeros_like(q))
    rows = w * terms.sum(1)
    share = 1.0 / max(count, 1) if reduction == "mean" else 1.0
    c = (w * share / temperature)[:, None]
    D = c * p
    D.scatter_add_(1, at, -c * q)
    dh = torch.zeros(T, H, dtype=torch.float64, device=dev)
    dh[take] = D @ W
    dW = D.t() @ h
    each = torch.zeros(T, dtype=torch.float64, device=dev)
    each[take] = rows
    each[bad] = math.nan
    loss = each if reduction == "none" else each.sum() * share
    if dtype is None:
        return loss, dh, dW
    sums = 6 * H + 16 if dtype == "fp32" else H + 8
    A = h.abs() @ W.abs().t() / temperature
    dz = sums * U * A
    most = dz.max(1, keepdim=True)[0] if len(take) else z.new_zeros(0, 1)
    dlse = most + (256 + 4 * lse.abs()) * U
    dterms = torch.where(q != 0, q * (dlse + dz.gather(1, at)) + 16 * U * q * (log_q.abs() + lse.abs() + zt.abs() + 1),
                         torch.zeros_like(q)) + 16 * U * terms.abs()
    # q itself: two roundings of its logit, the exponential, the sum, the quotient
    dterms = dterms + q * (lse - zt + log_q).abs() * (K + 64) * U * (1 + log_q.abs())
    drows = w.abs() * dterms.sum(1) + 4 * U * rows.abs()
    dp = p * (dz + dlse + 4 * U * (2 + z.abs() + lse.abs()))
    dD = c.abs() * dp + 8 * U * (c.abs() * p)
    if dtype == "bf16":
        most_p = p.max(1, keepdim=True)[0] if len(take) else p.new_zeros(0, 1)
        dD = dD + 1.01 * (U_BF16 ** d_terms + 2.0 ** -11) * (c.abs() * p) + 2.0 ** -39 * (c.abs() * most_p)
    own_q = torch.zeros_like(p).scatter_add_(1, at, q)
    dq = own_q * (K + 64) * U * (1 + (float(log_q.abs().max()) if log_q.numel() else 0.0))
    dD = dD + c.abs() * (dq + 4 * U * own_q) + (U_BF16 ** d_terms + 2 * U if dtype == "bf16" else U) * 1.01 * torch.where(own_q > 0, D.abs(), torch.zeros_like(D))
    tiny = 2.0 ** -126
    dD = dD + tiny * (2 * c.abs() + 2)
    last = U_BF16 if dtype == "bf16" else 2 * U
    deep = 6 if dtype == "fp32" else 1
    bh = torch.zeros(T, H, dtype=torch.float64, device=dev)
    bh[take] = (dD @ W.abs()) + (deep * V + 64) * U * (D.abs() @ W.abs()) + last * dh[take].abs() * 1.01 + tiny * (deep * V + 2)
    bW = dD.t() @ h.abs() + (deep * max(len(take), 1) + 64) * U * (D.abs().t() @ h.abs()) + last * dW.abs() * 1.01 + tiny * (deep * len(take) + 2)
    beach = torch.zeros(T, dtype=torch.float64, device=dev)
    beach[take] = drows
    bloss = beach if reduction == "none" else beach.sum() * share + 4 * U * loss.abs()
    return loss, dh, dW, bloss, bh, bW
