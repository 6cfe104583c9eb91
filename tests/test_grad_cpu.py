"""Gradient calls on the host: what they refuse, the workspace they ask for, and the oracle's own pins.

A refused call returns before any device work, so these run without a GPU; the
addresses here are never reached."""
import math

import numpy as np
import pytest

import allreduce_schedule_algorithms_amd as A
from oracle import grad as og

BAD = A.Status.AR_INVALID_ARGUMENT
BASE = 0x7000_0000_0000


def refused(call, status=BAD):
    with pytest.raises(A.ArError) as e:
        call()
    assert e.value.status == status
    return str(e.value)


def grads(*records):
    """Records (address, out, n[, dtype[, out_dtype]])."""
    return A.marshal_grads([(r + ("fp32", "fp32"))[:5] if len(r) < 5 else r for r in records])


def clip(**kw):
    kw.setdefault("max_norm", 1.0)
    kw.setdefault("total", BASE - 4096)
    return A.make_clip(**kw)


GOOD = (BASE, 0, 100)


@pytest.mark.parametrize("kw", [dict(norm=2), dict(norm=-1), dict(workspace=BASE + 8, workspace_bytes=1 << 20),
                                dict(total=BASE + 2), dict(each=BASE + 1), dict(total=None)])
def test_norm_refuses(kw):
    refused(lambda: A.ar_grad_norm(grads(GOOD), clip(**kw)))


def test_norm_takes_no_known_norm():
    refused(lambda: A.ar_grad_norm(grads(GOOD), clip(known=BASE - 64)))


@pytest.mark.parametrize("kw", [dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1e-6), dict(eps=math.nan),
                                dict(eps=math.inf), dict(norm=7), dict(known=BASE - 64),
                                dict(known=BASE - 64, total=None, each=BASE - 256), dict(known=BASE - 63, total=None)])
def test_clip_refuses(kw):
    refused(lambda: A.ar_grad_clip(grads(GOOD), clip(**kw)))


@pytest.mark.parametrize("rec", [
    (0, 0, 5), (BASE, 0, 5, "int32", "fp32"), (BASE, 0, 5, 9, 1), (BASE + 2, 0, 5), (BASE + 1, 0, 5, "bf16", "bf16"),
    (BASE, 0, 1 << 48), (BASE, 0, (1 << 64) - 1)])
def test_bad_tensors(rec):
    refused(lambda: A.ar_grad_norm(grads(rec), clip()))
    refused(lambda: A.ar_grad_clip(grads(rec), clip()))


@pytest.mark.parametrize("rec", [
    (BASE, BASE + 4096, 5, "fp32", "int32"), (BASE, BASE + 4098, 5, "fp32", "fp32"),
    (BASE, BASE, 5, "fp32", "bf16"),               # in place with another type
    (BASE, BASE + 4, 5, "fp32", "fp32"),           # shifted onto itself
    (BASE + 16, BASE, 5, "bf16", "fp32"),
    (BASE, BASE + 396, 100, "fp32", "bf16")])
def test_bad_outputs(rec):
    refused(lambda: A.ar_grad_clip(grads(rec), clip()))


def test_overlapping_tensors():
    a, b = (BASE, 0, 100), (BASE + 396, 0, 100)
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads(a, b), clip()))
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads(b, a), clip()))
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads(a, a), clip()))
    # a long tensor around a short one, not a neighbour in the order of addresses
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads((BASE, 0, 1000), (BASE + 40, 0, 0), (BASE + 80, 0, 1),
                                                             (BASE + 4000, 0, 8)), clip()))
    # one tensor's output on another's data, and two outputs on one place
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads((BASE, BASE + 8192, 100), (BASE + 8192, BASE + 16384, 100)), clip()))
    assert "overlap" in refused(lambda: A.ar_grad_clip(grads((BASE, BASE + 8192, 100), (BASE + 4096, BASE + 8192, 100)), clip()))


@pytest.mark.parametrize("known", [BASE, BASE + 4, BASE + 396])
def test_a_known_norm_may_not_lie_in_what_is_written(known):
    c = clip(known=known, total=None)
    for rec in (GOOD, (BASE, BASE, 100), (BASE + 8192, BASE, 100), (BASE + 8192, BASE, 200, "fp32", "bf16")):
        for records in ([rec], [(BASE + 4096, 0, 0), (BASE + 16384, 0, 7), rec]):
            assert "known" in refused(lambda: A.ar_grad_clip(grads(*records), c))
            assert "known" in refused(lambda: A.ar_grad_workspace_bytes(grads(*records), c))


@pytest.mark.parametrize("known", [BASE - 4, BASE + 400, BASE + 8192])
def test_a_known_norm_beside_what_is_written(known):
    # one in front, one behind, and one in a gradient that the call only reads
    empty = (BASE, known + 2, 0, "fp32", "bf16")
    assert A.ar_grad_workspace_bytes(grads((BASE + 8192, BASE, 100), empty), clip(known=known, total=None)) == 0


def test_counts():
    assert "count" in refused(lambda: A._ar._check(A._ar.lib.ar_grad_norm(None, -1, clip(), None)))
    assert "count" in refused(lambda: A._ar._check(A._ar.lib.ar_grad_norm(BASE, A.AR_MAX_GRADS + 1, clip(), None)))
    assert "NULL" in refused(lambda: A._ar._check(A._ar.lib.ar_grad_norm(None, 1, clip(), None)))
    assert "NULL" in refused(lambda: A._ar._check(A._ar.lib.ar_grad_clip(GOOD and grads(GOOD).address, 1, None, None)))


def rank_ptrs(P, n, elt=4, buckets=1, gap=256):
    step = n * elt + gap
    return [BASE + i * step // elt * elt for i in range(P * buckets)]


@pytest.mark.parametrize("kw", [dict(P=0), dict(P=257), dict(dtype="int32"), dict(dtype=5), dict(op="max"), dict(op=9),
                                dict(collective="all_gather"), dict(collective=-1), dict(n=[-1]), dict(n=[1 << 48]),
                                dict(max_norm=-1.0), dict(known=BASE - 64), dict(known=BASE - 64, total=None)])
def test_allreduce_clip_refuses(kw):
    c = clip(**{k: kw[k] for k in ("max_norm", "known", "total") if k in kw})
    a = dict(P=4, dtype="fp32", op="sum", collective="allreduce", n=[100])
    a.update({k: v for k, v in kw.items() if k in a})
    refused(lambda: A.ar_allreduce_clip(rank_ptrs(4, 100), a["n"], a["P"], a["dtype"], a["op"], a["collective"], c))


def test_allreduce_clip_buffers():
    def go(bufs, n=(100,), P=4, dtype="fp32"):
        return refused(lambda: A.ar_allreduce_clip(bufs, list(n), P, dtype, "sum", "allreduce", clip()))
    ok = rank_ptrs(4, 100)
    assert "NULL" in go(ok[:3] + [0])
    assert "aligned" in go(ok[:3] + [ok[3] + 2])
    assert "overlap" in go(ok[:3] + [ok[0]])
    assert "overlap" in go(ok[:3] + [ok[0] + 396])
    # buckets of one call may not share memory either
    assert "overlap" in go(ok + [p + 200 for p in ok], n=(100, 100))
    many = A.AR_MAX_GRADS // 4 + 1
    refused(lambda: A.ar_allreduce_clip_workspace_bytes([1] * many, 4, "fp32", "sum", "allreduce", clip()))


def test_workspace_bytes():
    # one workgroup takes a few small tensors and needs none
    assert A.ar_grad_workspace_bytes(grads(GOOD), clip()) == 0
    one = A.ar_grad_workspace_bytes(grads((BASE, 0, 200_000)), clip())
    assert 0 < one <= 4096
    # a partial for every workgroup, or for every item where the tensors' own norms are asked for
    sizes = [1000] * 5000
    many = grads(*[(BASE + i * 4096, 0, n) for i, n in enumerate(sizes)])
    assert one < A.ar_grad_workspace_bytes(many, clip()) < 1 << 16
    assert A.ar_grad_workspace_bytes(many, clip(each=BASE - (1 << 20))) >= 8 * 5000
    for each in (None, BASE - 256):
        assert A.ar_grad_workspace_bytes(grads((BASE, 0, 1 << 40)), clip(each=each)) < 1 << 20
    assert A.ar_grad_workspace_bytes(grads((BASE, 0, 200_000)), clip(known=BASE - 64, total=None)) == 0
    args = (8, "bf16", "sum")
    assert A.ar_allreduce_clip_workspace_bytes([106], *args, "allreduce", clip()) == 0
    n = 10_000
    assert 0 < A.ar_allreduce_clip_workspace_bytes([n, n], *args, "allreduce", clip()) < 1 << 16
    assert A.ar_allreduce_clip_workspace_bytes([n, n], *args, "reduce_scatter", clip()) >= 2 * n * 2  # lower halves of the sums


@pytest.mark.parametrize("total", [1 << 40, 1 << 46, 1 << 47, (1 << 48) - 1])
def test_items_with_own_norms_stay_countable(total):
    """A kernel counts an item's elements in 32 bits: a call has total / (2^31 - 1) items or more, and with own norms
    each of them has four 8-byte partials."""
    least = 4 * 8 * -(-total // (2 ** 31 - 1))
    c = clip(each=BASE - 256)
    assert A.ar_grad_workspace_bytes(grads((BASE, 0, total)), c) >= least
    # the same memory several times over: a norm only reads it
    assert A.ar_grad_workspace_bytes(grads(*[(BASE, 0, total // 1024)] * 1024), c) >= least * 1023 // 1024
    assert A.ar_allreduce_clip_workspace_bytes([total], 2, "fp32", "sum", "allreduce", c) >= least


def test_torch_side_refuses_host_tensors():
    import torch
    t = torch.zeros(4)
    for call in (lambda: A.grad_norm([t]), lambda: A.grad_clip([t], 1.0), lambda: A.allreduce_clip([t, t.clone()], 1.0),
                 lambda: A.allreduce_clip([], 1.0), lambda: A.allreduce_clip([[]], 1.0),
                 lambda: A.allreduce_clip([[t], [t, t]], 1.0), lambda: A.grad_clip([], 1.0, out=[t]),
                 lambda: A.grad_clip([t], 1.0, out=[])):
        refused(call)


# ---- the oracle ----
def test_oracle_norms():
    a, b = np.array([3.0, 0.0], np.float32), np.array([0.0, 4.0], np.float32)
    total, each = og.norms([a, b], "l2")
    assert total == 5.0 and list(each) == [3.0, 4.0]
    assert og.norms([a, b], "max")[0] == 4.0
    assert og.norms([np.float32([3e38, 3e38])], "l2")[0] == pytest.approx(4.2426406e38, rel=1e-7)
    assert og.norms([np.float32([1e-40])], "l2")[0] == float(np.float32(1e-40))
    assert math.isnan(og.norms([np.float32([1, math.nan, math.inf])], "max")[0])
    assert og.norms([], "l2")[0] == 0.0
    assert og.norms([np.array([0x3f80, 0xbf80], np.uint16)], "l2")[0] == math.sqrt(2)


def test_oracle_factor():
    assert og.factor(0.5, 1.0, 0.0) == 1.0 and og.factor(1.0, 1.0, 0.0) == 1.0
    assert og.factor(4.0, 1.0, 0.0) == 0.25 and og.factor(3.0, 1.0, 1.0) == 0.25
    assert og.factor(math.inf, 1.0, 0.0) == 0.0 and og.factor(math.inf, math.inf, 0.0) == 1.0
    assert math.isnan(og.factor(math.nan, 1.0, 0.0)) and og.factor(0.0, 0.0, 0.0) == 1.0


def test_oracle_combine_in_rank_order():
    x = np.float32([[1e8], [1.0], [-1e8], [1.0]])
    assert og.combine(x, "sum")[0] == 1.0  # ((1e8 + 1) - 1e8) + 1 with 1e8 + 1 rounded to 1e8
    assert og.combine(x, "avg")[0] == np.float32(0.25)
