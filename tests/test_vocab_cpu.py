"""Losses over a vocabulary on the host: what the calls refuse, the workspace they ask for, and the oracle's own pins.

A refused call returns before any device work, so these run without a GPU; the addresses here are never reached."""
import ctypes as C
import math

import pytest
import torch

import allreduce_schedule_algorithms_amd as A
from oracle import vocab as ov

BAD = A.Status.AR_INVALID_ARGUMENT
BASE = 0x7000_0000_0000
GAP = 1 << 32


def refused(call, status=BAD):
    with pytest.raises(A.ArError) as e:
        call()
    assert e.value.status == status
    return str(e.value)


def call(pieces=None, **kw):
    T, H = kw.pop("T", 8), kw.pop("H", 64)
    if pieces is None:
        pieces = [(BASE + 4 * GAP, BASE + 5 * GAP, 100, H, H), (BASE + 6 * GAP, BASE + 7 * GAP, 60, H, H)]
    args = dict(T=T, H=H, dtype="bf16", hidden=BASE, ld=H, pieces=pieces, ids=BASE + GAP, loss=BASE + 2 * GAP,
                dh=BASE + 3 * GAP, dh_ld=H, workspace=BASE + 8 * GAP, workspace_bytes=1 << 30)
    args.update(kw)
    return A.make_vocab(**args)


TEACHER = dict(top=4, ids_ld=4, logits=BASE + 9 * GAP, logits_ld=4)


def both(c):
    return [refused(lambda: A.ar_vocab_loss(c)), refused(lambda: A.ar_vocab_loss_grad(c))]


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 30), dict(H=0), dict(H=65537), dict(dtype="int32"), dict(dtype=9), dict(hidden=None),
    dict(hidden=BASE + 1), dict(ld=63), dict(ld=1 << 29), dict(ids=None), dict(ids=BASE + GAP + 4), dict(ids_bytes=2),
    dict(loss=None), dict(loss=BASE + 2 * GAP + 2), dict(temperature=0.0), dict(temperature=-1.0),
    dict(temperature=math.nan), dict(temperature=math.inf), dict(temperature=1e-45), dict(reduction=3),
    dict(reduction=-1), dict(top=-1), dict(top=1025, ids_ld=1025, logits=BASE + 9 * GAP, logits_ld=1025),
    dict(token_weights=BASE + 10 * GAP + 2), dict(workspace=BASE + 8 * GAP + 8), dict(pieces=[]),
    dict(TEACHER, ids_ld=3), dict(TEACHER, logits_ld=3), dict(TEACHER, logits=None), dict(TEACHER, logits_dtype="int32"),
    dict(TEACHER, logits=BASE + 9 * GAP + 2)])
def test_refused(kw):
    both(call(**kw))


@pytest.mark.parametrize("piece", [
    (None, BASE, 10, 64, 64), (BASE + 4 * GAP + 1, BASE, 10, 64, 64), (BASE + 4 * GAP, BASE, -1, 64, 64),
    (BASE + 4 * GAP, BASE, 10, 63, 64), (BASE + 4 * GAP, BASE, 0, 64, 64), (BASE + 4 * GAP, BASE, (1 << 20) + 1, 64, 64)])
def test_bad_pieces(piece):
    both(call(pieces=[piece]))


def test_a_vocabulary_that_is_too_large_or_too_many_ranks():
    half = (BASE + 4 * GAP, BASE + 5 * GAP, 1 << 19, 64, 64)
    other = (BASE + 6 * GAP, BASE + 7 * GAP, (1 << 19) + 1, 64, 64)
    assert "2^20" in both(call(pieces=[half, other]))[0]
    both(call(pieces=[(BASE + 4 * GAP, None, 0, 64, 64)] * 257))


@pytest.mark.parametrize("kw", [
    dict(dh=None), dict(dh=BASE + 3 * GAP + 1), dict(dh_ld=63), dict(dh=BASE), dict(dh=BASE + 64),
    dict(dh=BASE + 4 * GAP), dict(dh=BASE + GAP), dict(dh=BASE + 2 * GAP), dict(dh=BASE + 8 * GAP)])
def test_gradients_refuse(kw):
    refused(lambda: A.ar_vocab_loss_grad(call(**kw)))


@pytest.mark.parametrize("dw", [None, BASE + 5 * GAP + 1, BASE, BASE + 4 * GAP, BASE + 6 * GAP, BASE + 7 * GAP, BASE + 3 * GAP])
def test_piece_gradients_refuse(dw):
    pieces = [(BASE + 4 * GAP, dw, 100, 64, 64), (BASE + 6 * GAP, BASE + 7 * GAP, 60, 64, 64)]
    refused(lambda: A.ar_vocab_loss_grad(call(pieces=pieces)))


def test_loss_may_not_lie_in_an_input():
    both(call(loss=BASE + 8))
    both(call(loss=BASE + GAP + 4, ids_bytes=4))


@pytest.mark.parametrize("kw", [dict(), TEACHER, dict(dtype="fp32", ld=65, H=65, dh_ld=65,
                                                      pieces=[(BASE + 4 * GAP, BASE + 5 * GAP, 100, 65, 65)])])
def test_workspace(kw):
    need = {}
    for grad in (False, True):
        c = call(**kw)
        need[grad] = A.ar_vocab_workspace_bytes(c, grad)
        run = A.ar_vocab_loss_grad if grad else A.ar_vocab_loss
        for given in (dict(workspace_bytes=need[grad] - 1), dict(workspace=None, workspace_bytes=0)):
            message = refused(lambda: run(call(**dict(kw, **given))), A.Status.AR_WORKSPACE_TOO_SMALL)
            assert str(need[grad]) in message
    assert 0 < need[False] <= need[True]


def test_workspace_is_bounded_in_the_tokens():
    def need(T):
        return A.ar_vocab_workspace_bytes(call(T=T, pieces=[(BASE + 4 * GAP, BASE + 5 * GAP, 131072, 64, 64)]), True)
    # 128 bytes of hidden states, an id of 16 and a few more a token, once the logits' 4 GiB are reached
    assert need(1 << 22) - need(1 << 21) < (1 << 21) * 200
    assert need(1 << 22) < 7 << 30


def test_pointers_do_not_count_for_the_workspace_but_by_their_alignment():
    def at(w, T=100):
        return A.ar_vocab_workspace_bytes(call(T=T, pieces=[(w, None, 100, 64, 64)], hidden=None, ids=None, loss=None, dh=None))
    assert at(None) == at(BASE) < at(BASE + 2)
    assert at(BASE, 64) == at(BASE + 2, 64)  # few rows: read in place at any address


def test_null_arguments():
    lib = A._ar.lib
    assert lib.ar_vocab_loss(None, None) == BAD
    assert lib.ar_vocab_loss_grad(None, None) == BAD
    assert lib.ar_vocab_workspace_bytes(C.byref(call()), 1, None) == BAD
    c = call()
    c.pieces = None
    both(c)


def cpu_tensors(T=3, H=4, V=5):
    return torch.zeros(T, H), torch.zeros(V, H), torch.zeros(T, dtype=torch.long)


def test_python_refuses_what_is_not_on_a_gpu():
    h, w, y = cpu_tensors()
    for f in (A.vocab_loss, A.vocab_loss_grad):
        refused(lambda: f(h, w, y))
        refused(lambda: f(h, [w, w], y))
        refused(lambda: f(None, w, y))
    for f in (A.distill_loss, A.distill_loss_grad):
        refused(lambda: f(h, w, torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.long)))
        refused(lambda: f(h, w, None, torch.zeros(3, 2, dtype=torch.long)))


# ---- the oracle's pins ----
def example(top, seed=0, T=5, H=3, V=7):
    g = torch.Generator().manual_seed(seed)
    h, w = torch.randn(T, H, generator=g, dtype=torch.float64), torch.randn(V, H, generator=g, dtype=torch.float64)
    weights = torch.rand(T, generator=g) + 0.5
    if not top:
        ids = torch.randint(0, V, (T,), generator=g)
        ids[1] = -100
        return h, w, ids, None, weights
    ids = torch.randint(0, V, (T, top), generator=g)
    ids[0, 0] = ids[0, top - 1]  # the same id twice
    ids[1] = -1
    ids[2, 1:] = -1
    return h, w, ids, torch.randn(T, top, generator=g, dtype=torch.float64), weights


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_gradients_are_the_losses_differences(top, reduction):
    h, w, ids, logits, weights = example(top)
    kw = dict(reduction=reduction, temperature=1.3, token_weights=weights)
    loss, dh, dw = ov.loss_and_gradients(h, w, ids, logits, **kw)
    step = 1e-5
    for x, d in ((h, dh), (w, dw)):
        for i in range(x.numel()):
            at = x.view(-1)
            keep = float(at[i])
            at[i] = keep + step
            up = float(ov.loss_and_gradients(h, w, ids, logits, **kw)[0])
            at[i] = keep - step
            down = float(ov.loss_and_gradients(h, w, ids, logits, **kw)[0])
            at[i] = keep
            # central differences: a third derivative below 10^3 times step^2 / 6, and 2^-52 of the loss over the step
            assert abs((up - down) / (2 * step) - float(d.view(-1)[i])) < 1e-7


def test_cross_entropy_by_hand():
    h, w = torch.tensor([[1.0], [2.0]]), torch.tensor([[0.0], [math.log(3.0)]])
    loss, dh, dw = ov.loss_and_gradients(h, w, torch.tensor([1, -100]))
    # logits 0 and log 3: p = 1/4, 3/4
    assert float(loss) == pytest.approx(math.log(4 / 3), rel=1e-6)
    assert dh.tolist() == [[pytest.approx(-0.25 * math.log(3), rel=1e-6)], [0.0]]
    assert dw.tolist() == [[pytest.approx(0.25)], [pytest.approx(-0.25)]]


def test_distillation_of_the_student_itself_is_nothing():
    g = torch.Generator().manual_seed(1)
    h, w = torch.randn(4, 3, generator=g, dtype=torch.float64), torch.randn(6, 3, generator=g, dtype=torch.float64)
    ids = torch.stack([torch.randperm(6, generator=g) for _ in range(4)])
    logits = (h @ w.t()).gather(1, ids)
    loss, dh, dw = ov.loss_and_gradients(h, w, ids, logits, temperature=2.0)
    assert abs(float(loss)) < 1e-15 and float(dh.abs().max()) < 1e-15 and float(dw.abs().max()) < 1e-15


def test_a_single_entry_is_cross_entropy():
    h, w, ids, _, weights = example(0)
    ids[1] = 2
    a = ov.loss_and_gradients(h, w, ids, token_weights=weights)
    b = ov.loss_and_gradients(h, w, ids[:, None], torch.randn(5, 1, dtype=torch.float64), token_weights=weights)
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-14, atol=1e-16)


@pytest.mark.parametrize("top", [0, 3])
def test_a_mistake_in_the_oracle_shows(top):
    """The bounds are tight enough to tell a gradient without its own ids' part."""
    h, w, ids, logits, _ = example(top, T=5, H=8, V=40)
    loss, dh, dw, bl, bh, bw = ov.loss_and_gradients(h, w, ids, logits, dtype="bf16")
    kept = [0, 2, 3, 4]
    wrong = ov.loss_and_gradients(h, w, torch.where(ids < 0, ids, (ids + 1).clamp(max=39)), logits)
    assert float((wrong[0] - loss).abs()) > float(bl)
    assert bool(((wrong[1] - dh).abs() > bh)[kept].any(1).all())
    assert bool(((wrong[2] - dw).abs() > bw).any())


def test_a_temperature_whose_scale_is_infinite():
    """Logits are scaled by log2(e) / temperature: past the largest fp32 value it would make the difference of equal
    logits, 0, a NaN. 4.24e-39 is the smallest temperature that it does not."""
    largest = torch.finfo(torch.float32).max
    for t, fine in ((3e-39, False), (4.23e-39, False), (4.25e-39, True), (1e-38, True)):
        assert (float(torch.tensor(math.log2(math.e) / t, dtype=torch.float64)) <= largest) == fine
        if fine:
            assert A.ar_vocab_workspace_bytes(call(temperature=t), True) > 0
        else:
            assert all("log2(e)" in message for message in both(call(temperature=t)))
            refused(lambda: A.ar_vocab_workspace_bytes(call(temperature=t), False))


@pytest.mark.parametrize("top,dtype", [(0, "bf16"), (3, "fp32"), (64, "bf16"), (1024, "bf16"), (1024, "fp32")])
@pytest.mark.parametrize("rows", [100, 131072])
@pytest.mark.parametrize("grad", [False, True])
def test_what_of_the_workspace_grows_with_the_tokens(top, dtype, rows, grad):
    """4 GiB of logits, ids' logits and statistics; a token's hidden states, ids and some words, as ar.h lists them; and
    partial gradients of at most 512 MiB beside 4 bytes an element of W."""
    kw = dict(TEACHER, top=top, ids_ld=top, logits_ld=top) if top else {}
    ids = max(4, (top + 3) // 4 * 4)

    def need(T):
        return A.ar_vocab_workspace_bytes(call(T=T, dtype=dtype, pieces=[(BASE + 4 * GAP, BASE + 5 * GAP, rows, 64, 64)], **kw), grad)
    per = 64 * (6 if dtype == "fp32" else 2) + ids * (8 if top > 4 else 4) + 90
    terms = rows * 64 * 6 if dtype == "fp32" else 0
    for T in (1 << 16, 1 << 21, 1 << 24):
        assert need(T) <= (4 << 30) + T * per + terms + (512 << 20) + (rows + 255) * 64 * 4 + (1 << 20)


@pytest.mark.parametrize("lost", [None, 0, 1, 2, 3, 4, 5])
def test_a_lost_product_of_terms_shows(lost):
    """fp32 operands as three bf16 terms, and the six products that a call sums, smallest first: within 8 U of the value,
    and past it (and past what the GPU tests allow two of them, 10 U of both) where one is left out."""
    g = torch.Generator().manual_seed(2)
    x, y = [1 + torch.rand(2000, generator=g) for _ in range(2)]

    def terms(v):
        out = []
        for _ in range(3):
            out.append(v.bfloat16().float())
            v = v - out[-1]
        assert not bool(v.any())
        return out
    a, b = terms(x), terms(y)
    total = torch.zeros(2000)
    for i, (p, q) in enumerate([(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]):
        if i != lost:
            total += a[p] * b[q]
    exact = x.double() * y.double()
    off = ((total.double() - exact).abs() / exact).max()
    assert float(off) <= 8 * ov.U if lost is None else float(off) > 20 * ov.U
