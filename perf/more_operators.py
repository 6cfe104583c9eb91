"""Losses over a vocabulary that ranks hold in pieces, with their gradients: the cases that are measured.

Two operators on a model's last hidden states h [T, H] and an output matrix W [V, H] whose rows (the vocabulary)
lie in P pieces, one per rank, as one call's list of tensors:

* ``vocab_loss``    softmax cross entropy: with z = h W^T / temperature and target y_t,
                    loss_t = log(sum_v exp z_tv) - z_ty; rows of target -100 are left out;
* ``distill_loss``  distillation from a teacher's top logits: q_t = softmax of the teacher's K logits / temperature,
                    over the entries whose id is not negative; loss_t = sum_k q_tk (log q_tk - log p_t,id(k)), p_t the
                    softmax of z_t over the whole vocabulary; rows without entries are left out.

Each is measured as the loss alone and as the loss with d/dh and d/dW. "mean" divides by the rows that are not left
out; "none" returns every row's loss (0 where it is left out), and the gradients of their sum.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
IGNORE = -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(op, name=None, **kw):
    case = dict(op=op, grad=False, dtype="bf16", tokens=64, width=256, vocab=1000, pieces=1, odd=False, left_out=0.0,
                top=0, temperature=1.0, reduction="mean")
    case.update(kw)
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # a small probe's loss, read once a step: latency
        _case("vocab_loss", "loss_fp32_small", dtype="fp32", tokens=16, width=64, vocab=512),
        # scoring a few tokens' likelihood: the output matrix is read once, for 8 rows
        _case("vocab_loss", "loss_bf16_8_tokens", tokens=8, width=2048, vocab=32000, pieces=8, reduction="none"),
        # evaluation: a batch's per-token losses, a quarter of it padding, the vocabulary on 8 ranks
        _case("vocab_loss", "loss_bf16_eval", tokens=4096, width=2048, vocab=32000, pieces=8, left_out=0.25,
              reduction="none"),
        # ragged pieces in fp32, rows with gaps between them
        _case("vocab_loss", "loss_fp32_odd", dtype="fp32", tokens=1001, width=601, vocab=20011, pieces=3, odd=True),
        # a training step of a small head on two ranks: latency
        _case("vocab_loss", "grad_bf16_small", grad=True, tokens=48, width=256, vocab=1000, pieces=2),
        # a training step where prompts carry no loss: half of the rows are left out
        _case("vocab_loss", "grad_bf16_step", grad=True, tokens=8192, width=2048, vocab=32000, left_out=0.5),
        # the largest: a long batch against a large vocabulary on 8 ranks
        _case("vocab_loss", "grad_bf16_large", grad=True, tokens=8192, width=4096, vocab=128000, pieces=8),
        # fp32 training
        _case("vocab_loss", "grad_fp32", grad=True, dtype="fp32", tokens=2048, width=1024, vocab=32000),
        # the distance to a teacher, logged in evaluation
        _case("distill_loss", "distill_bf16_eval", tokens=1024, width=2048, vocab=32000, top=32, pieces=4,
              reduction="none"),
        # a small student: latency
        _case("distill_loss", "distill_grad_fp32_small", grad=True, dtype="fp32", tokens=32, width=128, vocab=800, top=8,
              temperature=2.0),
        # a student's training step against 64 logits a token
        _case("distill_loss", "distill_grad_bf16", grad=True, tokens=4096, width=2048, vocab=50000, top=64, pieces=4,
              temperature=2.0, left_out=0.1),
        # ragged: lists of different lengths, odd width and vocabulary, rows with gaps
        _case("distill_loss", "distill_grad_bf16_odd", grad=True, tokens=777, width=1001, vocab=30011, top=17, pieces=3,
              odd=True, left_out=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["vocab_loss", "distill_loss"])
    grad = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    while True:
        tokens, width, vocab = _log(rng, 1, 16384), _log(rng, 32, 4096), _log(rng, 100, 131072)
        if rng.random() < 0.5:  # as configured models have them
            width = max(32, width // 64 * 64)
            vocab = max(128, vocab // 64 * 64)
        cost = tokens * width * vocab * (3 if grad else 1) * (4 if dtype == "fp32" else 1)
        if cost <= 8192 * 4096 * 128000 * 3:
            break
    return _case(op, grad=grad, dtype=dtype, tokens=tokens, width=width, vocab=vocab, pieces=rng.choice([1, 1, 2, 3, 8]),
                 odd=rng.random() < 0.3, left_out=rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]),
                 top=min(_log(rng, 1, 128), vocab) if op == "distill_loss" else 0,
                 temperature=rng.choice([1.0, 1.0, 2.0, 0.7]), reduction=rng.choice(["mean", "none"]))


def _pieces(case):
    """Rows of each rank's piece."""
    V, P = case["vocab"], case["pieces"]
    if not case["odd"]:
        part = -(-V // P)
        sizes = [min(part, V - p * part) for p in range(P)]
    else:
        sizes = [max(1, V // P - 5 * (p + 1)) for p in range(P - 1)]
        sizes.append(V - sum(sizes))
    return sizes


def _kept(case):
    """Rows that are not left out."""
    return case["tokens"] - int(case["tokens"] * case["left_out"])


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H, V, K, dtype = case["tokens"], case["width"], case["vocab"], case["top"], DTYPES[case["dtype"]]
    gap = 3 if case["odd"] else 0

    def rows(n):
        return torch.empty(n, H + gap, dtype=dtype, device="cuda").normal_(0, 1, generator=g)[:, :H]

    # logits of a spread of about 2, as a partly trained model has them
    weights = [rows(n).mul_(2 * case["temperature"] / math.sqrt(H)) for n in _pieces(case)]
    hidden = rows(T)
    # token frequencies fall off as in text
    frequent = torch.rand(T, generator=g, device="cuda").pow_(4).mul_(V).long().clamp_(max=V - 1)
    whole = torch.cat(weights)
    # the hidden states know about their targets: z_ty is about 6 above the others
    hidden.add_(whole[frequent], alpha=1.5 / case["temperature"])
    out = torch.randperm(T, generator=g, device="cuda")[: T - _kept(case)]
    state = dict(case=case, hidden=hidden, weights=weights)
    if not K:
        frequent[out] = IGNORE
        state["targets"] = frequent
        return state
    # one id from each of K strata of the vocabulary, in an order of its own, the target's first
    edges = torch.arange(K + 1, device="cuda") * V // K
    ids = edges[:-1] + (torch.rand(T, K, generator=g, device="cuda") * (edges[1:] - edges[:-1])).long()
    ids = torch.minimum(ids, edges[1:] - 1)
    own_stratum = torch.searchsorted(edges, frequent, right=True) - 1
    ids.scatter_(1, own_stratum[:, None], frequent[:, None])
    order = torch.rand(T, K, generator=g, device="cuda").scatter_(1, own_stratum[:, None], -1.0).argsort(1)
    ids = ids.gather(1, order)
    logits = torch.empty(T, K, device="cuda").normal_(0, 2, generator=g).sort(1, descending=True)[0]
    logits[:, 0] += 2
    if case["odd"]:  # lists end at different lengths
        lengths = 1 + (torch.rand(T, generator=g, device="cuda") * K).long()
        ids[torch.arange(K, device="cuda")[None, :] >= lengths[:, None]] = -1
    ids[out] = -1
    state["ids"], state["logits"] = ids, logits
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(state):
    import allreduce_schedule_algorithms_amd as A
    case = state["case"]
    kw = dict(reduction=case["reduction"], temperature=case["temperature"])
    args = (state["hidden"], state["weights"])
    args += (state["logits"], state["ids"]) if case["top"] else (state["targets"],)
    if not case["grad"]:
        return dict(loss=(A.distill_loss if case["top"] else A.vocab_loss)(*args, **kw))
    loss, d_hidden, d_weights = (A.distill_loss_grad if case["top"] else A.vocab_loss_grad)(*args, **kw)
    return dict(loss=loss, d_hidden=d_hidden, d_weights=d_weights)


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    h, w = state["hidden"].float(), torch.cat(state["weights"]).float()
    z = h @ w.t() / case["temperature"]
    top = z.max(1, keepdim=True)[0]
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if case["top"]:
        there = state["ids"] >= 0
        ids = torch.where(there, state["ids"], 0)
        kept = there.any(1)
        t = torch.where(there, state["logits"] / case["temperature"], -math.inf)
        high = torch.where(kept, t.max(1)[0], 0.0)[:, None]
        a = torch.exp(t - high)
        norm = torch.where(kept, a.sum(1), 1.0)[:, None]
        q = a / norm
        log_q = torch.where(q > 0, t - high - torch.log(norm), 0.0)
        losses = (q * (log_q - (z.gather(1, ids) - lse))).sum(1)
    else:
        kept = state["targets"] != IGNORE
        ids = torch.where(kept, state["targets"], 0)[:, None]
        q = kept.float()[:, None]
        losses = torch.where(kept, (lse - z.gather(1, ids))[:, 0], 0.0)
    share = torch.where(kept, 1.0, 0.0)
    if case["reduction"] == "mean":
        count = share.sum().clamp(min=1.0)
        share = share / count
        loss = losses.sum() / count
    else:
        loss = losses
    if not case["grad"]:
        return dict(loss=loss)
    d = e * (share[:, None] / total)
    d.scatter_add_(1, ids, -q * share[:, None])
    d /= case["temperature"]
    d_hidden = (d @ w).to(state["hidden"].dtype)
    d_weights = (d.t() @ h).to(state["hidden"].dtype)
    return dict(loss=loss, d_hidden=d_hidden, d_weights=list(d_weights.split(_pieces(case))))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if 2 * case["tokens"] * case["width"] * case["vocab"] * (3 if case["grad"] else 1) > 1.5e14:
        return None
    state = prepare(case, seed)
    T, V, tau, sizes = case["tokens"], case["vocab"], case["temperature"], _pieces(case)
    w64 = torch.cat([w.double() for w in state["weights"]])
    losses = torch.zeros(T, dtype=torch.float64, device="cuda")
    kept = (state["ids"] >= 0).any(1) if case["top"] else state["targets"] != IGNORE
    count = max(int(kept.sum()), 1)
    scale = 1.0 / count if case["reduction"] == "mean" else 1.0
    if case["grad"]:
        d_hidden = torch.zeros(T, case["width"], dtype=torch.float64, device="cuda")
        d_weight = torch.zeros_like(w64)
    piece = max(1, (1 << 28) // V)
    for rows in kept.nonzero()[:, 0].split(piece):
        h64 = state["hidden"][rows].double()
        log_p = torch.log_softmax(torch.matmul(h64, w64.t()).div_(tau), dim=1)
        want = torch.zeros_like(log_p)  # the teacher's distribution, or the target's
        if case["top"]:
            ids = state["ids"][rows]
            gone = ids < 0
            t = (state["logits"][rows].double() / tau).masked_fill(gone, -math.inf)
            q = torch.softmax(t, dim=1)
            log_q = torch.log_softmax(t, dim=1).masked_fill(q == 0, 0.0)
            at = ids.masked_fill(gone, 0)
            losses[rows] = (q * (log_q - log_p.gather(1, at))).sum(1)
            want.scatter_add_(1, at, q)
        else:
            at = state["targets"][rows][:, None]
            losses[rows] = -log_p.gather(1, at)[:, 0]
            want.scatter_(1, at, 1.0)
        if case["grad"]:
            d = log_p.exp_().sub_(want).mul_(scale / tau)
            d_hidden[rows] = torch.matmul(d, w64)
            d_weight.addmm_(d.t(), h64)
        del log_p, want
    loss = losses.sum() / count if case["reduction"] == "mean" else losses
    if not case["grad"]:
        return dict(loss=loss)
    return dict(loss=loss, d_hidden=d_hidden, d_weights=list(d_weight.split(sizes)))


def work(case):
    e, T, H, V = 4 if case["dtype"] == "fp32" else 2, case["tokens"], case["width"], case["vocab"]
    kept = _kept(case)
    read = (kept + V) * H * e + T * (12 * case["top"] if case["top"] else 8)
    written = 4 if case["reduction"] == "mean" else 4 * T
    if case["grad"]:
        written += (T + V) * H * e
    return dict(bytes=read + written, flops=2 * kept * H * V * (3 if case["grad"] else 1))
