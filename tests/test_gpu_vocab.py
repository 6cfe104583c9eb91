"""Losses over a vocabulary in pieces on the GPU against their definition in 64 bits (oracle/vocab.py), within the
bounds that it derives for every element from the roundings of a call."""
import math

import pytest

from oracle import vocab as ov
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu

TYPES = ("bf16", "fp32")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    torch.cuda.set_device(0)


def lib():
    import allreduce_schedule_algorithms_amd as A
    return A


def of(dtype):
    torch = torch_mod()
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]


class Case:
    """Inputs on the GPU; gap: elements between the rows of every matrix, which hold NaN."""

    def __init__(self, T, H, pieces, dtype="bf16", top=0, seed=0, gap=0, scale=1.0, left_out=0.0, weights=False,
                 wide=True, logits_dtype="fp32", **kw):
        torch = torch_mod()
        g = torch.Generator(device="cuda").manual_seed(seed)
        V = sum(pieces)

        def matrix(n):
            big = torch.full((n, H + gap), math.nan, dtype=of(dtype), device="cuda")
            view = big[:, :H]
            if n:
                view.copy_(torch.randn(n, H, generator=g, device="cuda"))
            return view

        self.hidden = matrix(T)
        self.weight = [matrix(n) for n in pieces]
        for w in self.weight:
            w.mul_(2 * scale / math.sqrt(H))
        out = torch.rand(T, generator=g, device="cuda") < left_out
        self.logits = None
        if top:
            self.ids = torch.randint(0, V, (T, top), generator=g, device="cuda")
            self.ids[torch.rand(T, top, generator=g, device="cuda") < 0.2] = -1
            self.ids[out] = -7
            self.logits = (2 * torch.randn(T, top, generator=g, device="cuda")).to(of(logits_dtype))
        else:
            self.ids = torch.randint(0, V, (T,), generator=g, device="cuda")
            self.ids[out] = -100
        if not wide:
            self.ids = self.ids.int()
        self.kw = dict(kw)
        if weights:
            self.kw["token_weights"] = torch.randn(T, generator=g, device="cuda")
            self.kw["token_weights"][torch.rand(T, generator=g, device="cuda") < 0.2] = 0
        self.dtype = dtype

    def run(self, grad=True, **extra):
        A = lib()
        args = (self.hidden, self.weight) + ((self.ids,) if self.logits is None else (self.logits, self.ids))
        f = (A.vocab_loss_grad, A.distill_loss_grad) if grad else (A.vocab_loss, A.distill_loss)
        return f[self.logits is not None](*args, **{**self.kw, **extra})

    def want(self, dtype=True, **extra):
        torch = torch_mod()
        return ov.loss_and_gradients(self.hidden, torch.cat(self.weight), self.ids, self.logits,
                                     dtype=self.dtype if dtype else None, **{**self.kw, **extra})

    def check(self, got=None, **extra):
        torch = torch_mod()
        loss, dh, dw = got or self.run(**extra)
        alone = self.run(grad=False, **extra)
        torch.cuda.synchronize()
        want = self.want(**{k: v for k, v in extra.items() if k not in ("out_hidden", "out_weight", "workspace", "stream")})
        assert loss.dtype == torch.float32 and dh.dtype == of(self.dtype)
        assert [tuple(d.shape) for d in dw] == [tuple(w.shape) for w in self.weight]
        within(alone, want[0], want[3], "loss alone")
        within(loss, want[0], want[3], "loss")
        within(dh, want[1], want[4], "d_hidden")
        within(torch.cat(list(dw)), want[2], want[5], "d_weight")
        return loss, dh, dw


def within(got, want, bound, what):
    torch = torch_mod()
    got = got.double()
    assert got.shape == want.shape
    assert bool((torch.isnan(got) == torch.isnan(want)).all()), what
    off = torch.where(torch.isnan(want), torch.zeros_like(want), (got - want).abs() - bound)
    assert bool((off <= 0).all()), f"{what}: {float(off.max()):.3g} past its bound at {int(off.argmax())} of {want.numel()}"


def same(a, b):
    """The same bits, NaN too."""
    torch = torch_mod()
    flat = lambda r: [r[0], r[1]] + list(r[2])
    for x, y in zip(flat(a), flat(b)):
        i = {4: torch.int32, 2: torch.int16}[x.element_size()]
        assert torch.equal(x.contiguous().view(i), y.contiguous().view(i))


# T, H, pieces: single rows and elements, one row more or less than a tile or a slice, ranks without rows
SHAPES = [
    (1, 1, [1]), (1, 64, [2]), (2, 8, [1, 1]), (3, 5, [7]), (16, 64, [512]), (17, 40, [255, 257]), (63, 72, [100]),
    (64, 32, [256]), (65, 96, [0, 300, 0]), (129, 128, [1, 640, 3]), (200, 33, [999]), (257, 130, [384, 385]),
    (300, 264, [1500, 700]), (40, 1000, [65] * 5)]


@pytest.mark.parametrize("T,H,pieces", SHAPES)
@pytest.mark.parametrize("top", [0, 1, 5])
@pytest.mark.parametrize("dtype", TYPES)
def test_shapes(T, H, pieces, top, dtype):
    Case(T, H, pieces, dtype, top, seed=T + H, left_out=0.3 if T > 2 else 0.0).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("top", [0, 4, 9])
def test_reductions_weights_and_temperatures(dtype, reduction, top):
    Case(90, 48, [130, 200], dtype, top, seed=3, left_out=0.25, weights=True, reduction=reduction, temperature=0.6).check()


@pytest.mark.parametrize("gap", [1, 3, 8])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_apart(gap, dtype):
    """Gaps between rows hold NaN: nothing of them may come into a result."""
    Case(70, 64, [100, 90], dtype, seed=gap, gap=gap).check()
    Case(70, 61, [100, 90], dtype, top=3, seed=gap, gap=gap).check()


@pytest.mark.parametrize("offset", [0, 1, 2, 8])
def test_pieces_at_any_element(offset):
    torch = torch_mod()
    c = Case(40, 64, [96, 64], seed=offset)
    flat = torch.empty(160 * 64 + offset, dtype=torch.bfloat16, device="cuda")
    flat[offset:].view(160, 64).copy_(torch.cat(c.weight))
    c.weight = list(flat[offset:].view(160, 64).split([96, 64]))
    c.check()


@pytest.mark.parametrize("dtype,H", [("bf16", 64), ("bf16", 50), ("fp32", 33)])
def test_outputs_given(dtype, H):
    """Into rows with gaps at an odd element, which keep what is between them."""
    torch = torch_mod()
    c = Case(37, H, [70, 300], dtype, seed=8, left_out=0.2)
    want = c.run()

    def room(n):
        big = torch.full((n * (H + 5) + 3,), 7.0, dtype=of(dtype), device="cuda")
        return big, big[3:].view(n, H + 5)[:, :H]

    bigs, views = zip(*[room(n) for n in (37, 70, 300)])
    got = c.run(out_hidden=views[0], out_weight=list(views[1:]))
    torch.cuda.synchronize()
    assert got[1] is views[0] and got[2][1] is views[2]
    same(want, got)
    for big, n in zip(bigs, (37, 70, 300)):
        assert bool((big[:3] == 7).all()) and bool((big[3:].view(n, H + 5)[:, H:] == 7).all())


def test_a_single_tensor_as_the_output_matrix():
    torch = torch_mod()
    c = Case(20, 32, [50])
    loss, dh, dw = lib().vocab_loss_grad(c.hidden, c.weight[0], c.ids)
    assert isinstance(dw, torch.Tensor)
    same((loss, dh, [dw]), c.run())


@pytest.mark.parametrize("top", [0, 6])
def test_ids_of_32_bits_and_teachers_in_bf16(top):
    Case(50, 40, [90, 33], top=top, seed=2, wide=False, logits_dtype="bf16", left_out=0.1).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_the_large_tiles(dtype):
    """Enough outputs that every product runs on the largest tiles; and rows left out shorten the depth."""
    Case(777, 520, [20000, 5000, 31], dtype, seed=11, left_out=0.4).check()


def test_distillation_on_the_large_tiles():
    Case(600, 256, [30000], top=64, seed=12, left_out=0.1, temperature=2.0).check()


@pytest.mark.parametrize("top", [0, 2])
def test_the_medium_tiles(top):
    Case(400, 200, [3000], top=top, seed=13).check()


def test_the_most_teacher_entries():
    Case(9, 16, [2000], top=1024, seed=14).check()


@pytest.mark.parametrize("P", [64, 65, 130, 256])
def test_many_ranks(P):
    Case(30, 24, [1 + p % 5 for p in range(P)], seed=P).check()


@pytest.mark.parametrize("top", [0, 3, 8])
@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_left(top, dtype):
    torch = torch_mod()
    c = Case(33, 40, [60], dtype, top, left_out=1.1)
    c.hidden.fill_(math.nan)
    for reduction, zero in (("mean", 0), ("sum", 0), ("none", torch.zeros(33))):
        loss, dh, dw = c.run(reduction=reduction)
        assert bool((loss.cpu() == zero).all()) and not bool(dh.any()) and not bool(dw[0].any())
        assert bool((c.run(False, reduction=reduction).cpu() == zero).all())


@pytest.mark.parametrize("top", [0, 3])
def test_no_tokens(top):
    torch = torch_mod()
    A = lib()
    w = torch.randn(50, 16, device="cuda")
    h, ids, logits = torch.empty(0, 16, device="cuda"), torch.empty((0, top) if top else 0, dtype=torch.long, device="cuda"), torch.empty(0, top, device="cuda")
    loss, dh, dw = A.distill_loss_grad(h, w, logits, ids) if top else A.vocab_loss_grad(h, w, ids)
    assert float(loss) == 0 and dh.shape == (0, 16) and not bool(dw.any())
    assert (A.distill_loss(h, w, logits, ids, "none") if top else A.vocab_loss(h, w, ids, "none")).shape == (0,)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [0, 4])
def test_what_is_masked_is_not_read(dtype, top):
    """NaN and infinities in rows that are left out or weigh nothing, and in the logits of absent entries."""
    torch = torch_mod()
    c = Case(80, 48, [200], dtype, top, seed=5, left_out=0.3, weights=True)
    want = c.run()
    if top:
        gone = (c.ids < 0).all(1)
        c.logits[c.ids < 0] = math.nan
    else:
        gone = c.ids == -100
    c.hidden[gone | (c.kw["token_weights"] == 0)] = math.inf
    same(want, c.run())


@pytest.mark.parametrize("top", [0, 4])
def test_ids_outside_the_vocabulary(top):
    torch = torch_mod()
    c = Case(40, 32, [70, 30], top=top, seed=6, left_out=0.1)
    bad = [3, 17]
    c.ids[3] = 100
    c.ids[17] = 1 << 40
    if not top:
        c.ids[20] = -1
        bad.append(20)
    c.check(reduction="none")
    loss, dh, dw = c.run()
    assert math.isnan(float(loss)) and math.isnan(float(c.run(False))) and not bool(dh[bad].any())
    want = c.want(reduction="mean")
    within(dh, want[1], want[4], "d_hidden")
    within(torch.cat(dw), want[2], want[5], "d_weight")


def test_teacher_lists():
    """The same id twice, entries of -infinity, a list of them alone, and a single entry."""
    torch = torch_mod()
    c = Case(6, 24, [40], top=5, seed=7)
    c.ids[:] = torch.tensor([[4, 4, 9, 4, 39], [1, 2, 3, 4, 5], [7, 7, 7, 7, 7], [0, -1, -1, -1, -1], [-1, -1, 12, -1, 13], [8, 9, 10, 11, 12]])
    c.logits[1, :3] = -math.inf
    c.logits[5] = -math.inf
    loss, dh, _ = c.check(reduction="none")
    assert float(loss[5]) == 0 and not bool(dh[5].any())
    c.check()


def test_a_teacher_that_is_not_finite():
    c = Case(5, 24, [40], top=3, seed=9, reduction="none")
    c.ids.clamp_(min=0)
    c.logits[1, 1] = math.nan
    c.logits[2, 2] = math.inf
    loss = c.run(False)
    assert [math.isnan(float(x)) for x in loss] == [False, True, True, False, False]


@pytest.mark.parametrize("dtype", TYPES)
def test_hidden_states_that_are_not_finite(dtype):
    torch = torch_mod()
    c = Case(40, 32, [300], dtype, seed=10, reduction="none")
    whole = c.run()
    c.hidden[7, 3] = math.nan
    c.hidden[11, 0] = math.inf
    loss, dh, dw = c.run()
    rows = [i for i in range(40) if i not in (7, 11)]
    assert bool(torch.isnan(loss[[7, 11]]).all()) and torch.equal(loss[rows], whole[0][rows])
    assert bool(torch.isnan(dh[[7, 11]]).all()) and torch.equal(dh[rows], whole[1][rows])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, 1e-6, 60.0, 3e3])
def test_magnitudes(dtype, scale):
    """From a uniform distribution to one that is a single id."""
    Case(60, 40, [500], dtype, seed=15, scale=scale).check()


def test_the_ends_of_the_range():
    """fp32 values whose bf16 rounding would be infinite, and those whose terms lie below the smallest normal value."""
    torch = torch_mod()
    A = lib()
    big = torch.tensor([[3.4e38, 0.0]], device="cuda")
    w = torch.tensor([[1e-38, 0.0], [0.0, 1.0]], device="cuda")
    loss = A.vocab_loss(big, w, torch.tensor([0], device="cuda"))
    want = ov.loss_and_gradients(big, w, torch.tensor([0], device="cuda"))[0]
    # An fp32 operand is a sum of bf16 terms, whose grid ends at 2^-133: w is off by 2^-134 at most, its logit by
    # 3.4e38 times that, and the loss by no more (with 2^-20 for the rest: logits of 3.4 and 0).
    assert abs(float(loss) - float(want)) < 3.4e38 * 2.0 ** -134 + 2.0 ** -20
    assert math.isfinite(float(loss))
    w[0, 0] = 1e-33  # all 24 bits lie above the grid's end: six roundings of 2^-24 of a loss of 340000, at most 16
    loss = A.vocab_loss(big, w, torch.tensor([1], device="cuda"))
    assert float(loss) == pytest.approx(float(ov.loss_and_gradients(big, w, torch.tensor([1], device="cuda"))[0]), rel=2.0 ** -20)


def test_the_same_bits_on_every_run():
    torch = torch_mod()
    for c in (Case(300, 256, [9000], seed=16, left_out=0.2), Case(100, 64, [700], "fp32", top=9, seed=17)):
        first = c.run()
        noise = torch.empty(1 << 26, device="cuda")
        for _ in range(3):
            noise.normal_()
            same(first, c.run())


@pytest.mark.parametrize("limit", [1, 3, 1000])
def test_launch_limit(limit):
    A = lib()
    cases = [Case(70, 64, [300, 30], "fp32", seed=18, left_out=0.3), Case(70, 64, [300, 30], top=6, seed=18)]
    prev = A.ar_set_launch_blocks(limit)
    try:
        for c in cases:
            c.check()
    finally:
        A.ar_set_launch_blocks(prev)


@pytest.mark.parametrize("top", [0, 6])
def test_captured(top):
    """A graph replays on new inputs, beside eager calls of the same sizes and of its own tensors."""
    torch = torch_mod()
    c = Case(50, 64, [400, 100], top=top, seed=19, left_out=0.2)
    other = Case(50, 64, [400, 100], top=top, seed=20, left_out=0.5)
    c.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c.run()
        graphs.append((graph, out))
    for turn in range(4):
        if turn % 2:
            c.hidden.copy_(other.hidden)
            c.ids.copy_(other.ids)
            if top:
                c.logits.copy_(other.logits)
        else:
            c.hidden.neg_()
        want = c.run()
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        c.run()
        for graph, out in graphs:
            torch.cuda.synchronize()
            same(want, out)


def test_streams():
    """Calls on two streams at once, one named by its number, with workspaces of their own."""
    torch = torch_mod()
    a, b = Case(200, 128, [3000], seed=21), Case(200, 128, [3000], seed=22, top=5)
    wa, wb = a.run(), b.run()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        ga, gb = a.run(stream=s), b.run(stream=t.cuda_stream)
    torch.cuda.synchronize()
    same(wa, ga)
    same(wb, gb)


def test_workspace_of_the_callers_own():
    torch = torch_mod()
    A = lib()
    c = Case(60, 64, [200, 100], seed=23)
    want = c.run()
    for grad in (True, False):
        call = A.make_vocab(60, 64, "bf16", c.hidden.data_ptr(), 64,
                            [(w.data_ptr(), None, w.shape[0], 64, 64) for w in c.weight], c.ids.data_ptr(), None, dh_ld=64)
        need = A.ar_vocab_workspace_bytes(call, grad)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
        got = c.run(grad, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((ws[need:] == 255).all())
        if grad:
            same(want, got)
        else:
            assert torch.equal(got, want[0])
        with pytest.raises(A.ArError) as e:
            c.run(grad, workspace=ws[:need - 1])
        assert e.value.status == A.Status.AR_WORKSPACE_TOO_SMALL


def test_refused_in_python():
    torch = torch_mod()
    A = lib()
    c = Case(10, 16, [20], seed=24)
    h, w, y = c.hidden, c.weight[0], c.ids
    lg, ids = torch.zeros(10, 3, device="cuda"), torch.zeros(10, 3, dtype=torch.long, device="cuda")
    bad = [
        lambda: A.vocab_loss(h.half(), w.half(), y), lambda: A.vocab_loss(h, w.float(), y), lambda: A.vocab_loss(h, w[:, :8], y),
        lambda: A.vocab_loss(h, w.cpu(), y), lambda: A.vocab_loss(h, w, y.cpu()), lambda: A.vocab_loss(h, w, y[:9]),
        lambda: A.vocab_loss(h, w, y.float()), lambda: A.vocab_loss(h, w, ids), lambda: A.vocab_loss(h.t().contiguous().t(), w, y),
        lambda: A.vocab_loss(h, w.t().contiguous().t(), y), lambda: A.vocab_loss(h, w, y, reduction="average"),
        lambda: A.vocab_loss(h, w, y, temperature=0.0), lambda: A.vocab_loss(h, w, y, token_weights=torch.ones(9, device="cuda")),
        lambda: A.vocab_loss(h, w, y, token_weights=torch.ones(10, device="cuda").double()), lambda: A.vocab_loss(h, [], y),
        lambda: A.vocab_loss(h, w, y, token_weights=[1.0] * 10),
        lambda: A.vocab_loss(h[:, :0], w[:, :0], y), lambda: A.vocab_loss(h[:1].expand(10, 16), w, y),
        lambda: A.vocab_loss(h[0], w, y), lambda: A.vocab_loss(h, w[:0], y),
        lambda: A.vocab_loss_grad(h, w, y, out_hidden=h), lambda: A.vocab_loss_grad(h, w, y, out_weight=w),
        lambda: A.vocab_loss_grad(h, w, y, out_hidden=torch.empty(10, 16, device="cuda")),
        lambda: A.vocab_loss_grad(h, w, y, out_weight=torch.empty_like(h)), lambda: A.vocab_loss_grad(h, [w], y, out_weight=[]),
        lambda: A.distill_loss(h, w, lg, ids[:, :2]), lambda: A.distill_loss(h, w, lg[:, :0], ids[:, :0]),
        lambda: A.distill_loss(h, w, lg, y), lambda: A.distill_loss(h, w, lg.half(), ids), lambda: A.distill_loss(h, w, None, ids),
        lambda: A.distill_loss(h, w, torch.zeros(10, 1025, device="cuda"), torch.zeros(10, 1025, dtype=torch.long, device="cuda")),
        lambda: A.vocab_loss(h, w, y, workspace=torch.empty(1 << 22, dtype=torch.uint8))]
    for f in bad:
        with pytest.raises(A.ArError) as e:
            f()
        assert e.value.status == A.Status.AR_INVALID_ARGUMENT


def test_written_outputs_are_known_to_autograd():
    torch = torch_mod()
    c = Case(10, 16, [20], seed=25)
    out = torch.empty_like(c.hidden)
    x = torch.ones(10, 16, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = (x * out).sum()
    c.run(out_hidden=out)
    with pytest.raises(RuntimeError):
        y.backward()


def test_gradients_are_the_losses_differences():
    """fp32, along random directions: the loss is off by its bound, a difference over 2 e by that over e, and central
    differences by e^2 / 6 of the third derivative along the direction."""
    torch = torch_mod()
    for top in (0, 3):
        c = Case(24, 16, [40], "fp32", top, seed=26, scale=0.5)
        want = c.want()
        _, dh, dw = c.run()
        g = torch.Generator(device="cuda").manual_seed(27)
        for x, d in ((c.hidden, dh), (c.weight[0], dw[0])):
            u = torch.randn(x.shape, generator=g, device="cuda")
            u /= u.norm()
            e = 2.0 ** -5
            keep = x.clone()
            x.copy_(keep + e * u)
            up = float(c.run(False))
            x.copy_(keep - e * u)
            down = float(c.run(False))
            x.copy_(keep)
            # third derivative: at most 2 |dz|^3 a row (a softmax's third cumulant), |dz| <= |other operand's rows|
            reach = max(float(c.weight[0].norm(dim=1).max()), float(c.hidden.norm(dim=1).max()))
            tol = 2 * float(want[3]) / e + e * e / 3 * reach ** 3 + 2.0 ** -20
            assert abs((up - down) / (2 * e) - float((u.double() * d.double()).sum())) < tol


def test_together():
    """A step of P data-parallel replicas of a head whose vocabulary lies on ranks: losses and gradients, averaged and
    clipped as buckets, and a second replica's gradients from a teacher."""
    torch = torch_mod()
    A = lib()
    cases = [Case(64, 48, [200, 150], "fp32", top=t, seed=30 + t, left_out=0.2) for t in (0, 0, 4)]
    for c in cases[1:]:
        c.weight = cases[0].weight
    grads = [c.run()[2] for c in cases]
    want = [c.want(False)[2] for c in cases]
    buckets = [[g[p] for g in grads] for p in range(2)]
    norm = A.allreduce_clip(buckets, 0.01, op="avg")
    mean = sum(want) / 3
    assert float(norm) == pytest.approx(float(mean.norm()), rel=1e-5)
    scale = min(1.0, 0.01 / (float(mean.norm()) + 1e-6))
    for g in grads:
        assert torch.allclose(torch.cat(g).double(), mean * scale, rtol=1e-4, atol=1e-8)


def test_tokens_in_chunks():
    """More logits than a call keeps at a time: gradients add up over the chunks."""
    torch = torch_mod()
    T, H, V = 40000, 32, 131072
    c = Case(T, H, [V - 1000, 1000], seed=31, left_out=0.1)
    loss, dh, dw = c.run(reduction="sum")
    alone = c.run(False, reduction="sum")
    W, h = torch.cat(c.weight).double(), c.hidden.double()
    kept = (c.ids != -100).nonzero()[:, 0]
    lse = torch.zeros(T, dtype=torch.float64, device="cuda")
    for rows in kept.split(2000):
        lse[rows] = torch.logsumexp(h[rows] @ W.t(), 1)
    zt = (h * W[c.ids.clamp(min=0)]).sum(1)
    want = float((lse - zt)[kept].sum())
    # every row's loss: the bounds of its logits (H + 8 roundings of up to 60), and 300 of its log-sum-exp
    assert abs(float(loss) - want) < T * 2.0 ** -24 * (60 * (H + 8) + 400)
    assert abs(float(alone) - want) < T * 2.0 ** -24 * (60 * (H + 8) + 400)
    cols = torch.cat([torch.arange(0, V, 1777, device="cuda"), torch.tensor([V - 1001, V - 1000, V - 1], device="cuda")])
    D = torch.exp(h[kept] @ W[cols].t() - lse[kept, None])
    own = c.ids[kept][:, None] == cols[None, :]
    bound = D * (2.02 * ov.U_BF16 + 4e-4) + own * 0.01
    D = D - own.double()
    want_w = D.t() @ h[kept]
    tol = bound.t() @ h[kept].abs() + 2.0 ** -24 * T * (D.abs().t() @ h[kept].abs()) + ov.U_BF16 * want_w.abs()
    within(torch.cat(dw)[cols], want_w, tol, "d_weight")
    some = kept[::997]
    D = torch.exp(h[some] @ W.t() - lse[some, None])
    bound = D * (2.02 * ov.U_BF16 + 4e-4)
    D[torch.arange(len(some)), c.ids[some]] -= 1
    bound[torch.arange(len(some)), c.ids[some]] += 0.01
    want_h = D @ W
    tol = bound @ W.abs() + 2.0 ** -24 * V * (D.abs() @ W.abs()) + ov.U_BF16 * want_h.abs()
    within(dh[some], want_h, tol, "d_hidden")
    assert not bool(dh[c.ids == -100].any())


def test_an_output_matrix_of_more_than_2_31_elements():
    torch = torch_mod()
    T, H, V = 5, 2112, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(32)
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02, generator=g)
    h = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([0, V - 1, V // 2, 123456, -100], device="cuda")
    loss, dh, dw = lib().vocab_loss_grad(h, w, ids, reduction="none")
    z = torch.cat([h.double() @ p.double().t() for p in w.split(1 << 17)], 1)
    p = torch.softmax(z, 1)
    want = torch.logsumexp(z, 1) - z.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    want[4] = 0
    # |h| |W| is below 60 for these; a log-sum-exp of 14
    assert bool(((loss.double() - want).abs() < 2.0 ** -24 * (60 * (H + 8) + 400)).all())
    p[torch.arange(4), ids[:4]] -= 1
    p[4] = 0
    rows = torch.tensor([0, 1, V // 2, V // 2 + 1, 123456, V - 2, V - 1], device="cuda")
    want_w = p[:, rows].t() @ h.double()
    tol = (p[:, rows].abs() * (2.02 * ov.U_BF16 + 0.02)).t() @ h.double().abs() + ov.U_BF16 * want_w.abs() + 1e-12
    within(dw[rows], want_w, tol, "d_weight")
    want_h = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want_h)
    for i, part in enumerate(w.split(1 << 17)):
        q = p[:, i << 17: (i + 1) << 17]
        want_h += q @ part.double()
        size += (q.abs() * (2.02 * ov.U_BF16 + 0.02)) @ part.double().abs()
    within(dh, want_h, size + ov.U_BF16 * want_h.abs(), "d_hidden")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_largest_vocabulary_with_lists_of_ids(dtype):
    """As many tiles of logits as there can be, whose ids are sorted."""
    Case(3, 16, [1 << 19, 1 << 18, 1 << 18], dtype, top=6, seed=33).check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [8, 9, 33, 64, 127, 128])
def test_rows_around_the_changes_of_kernel(dtype, T):
    """Rows packed by the first launch or their own, and up to 64 and 128 rows' tiles."""
    Case(T, 512, [700, 900], dtype, seed=34, left_out=0.2).check()
    Case(T, 511, [700, 900], dtype, top=5, seed=35, left_out=0.2).check()


def shifted(c, by):
    """The same case with all of its logits moved by `by` (over the temperature), through the last column."""
    c.hidden[:, -1] = 1
    for w in c.weight:
        w[:, -1] = by
    return c


@pytest.mark.parametrize("by", [-200.0, 200.0])
@pytest.mark.parametrize("top", [0, 3, 6])
@pytest.mark.parametrize("T", [16, 50, 100, 300])
@pytest.mark.parametrize("dtype", TYPES)
def test_logits_far_from_zero(dtype, T, top, by):
    """A softmax does not know of a shift: neither may the tiles that lie behind a piece's rows, of 64, 128 or 256 rows."""
    for pieces in ([100], [300], [41, 300], [65, 0, 1]):
        shifted(Case(T, 40, pieces, dtype, top, seed=36, left_out=0.1), by).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_logits_far_from_zero_over_many_tiles(dtype):
    shifted(Case(100, 64, [50257], dtype, top=3, seed=37, temperature=0.5), -60.0).check()


def test_a_tile_whose_logits_are_all_minus_infinity():
    """Rows of W that hold -infinity (the next smallest logits are below -89): no share of the distribution."""
    torch = torch_mod()
    for T in (20, 200):
        c = shifted(Case(T, 40, [400], seed=38, reduction="none"), -200.0)
        c.hidden[:, 0] = 1
        c.ids.fill_(7)
        want = lib().vocab_loss_grad(c.hidden, c.weight[0][:128], c.ids, "none")
        c.weight[0][128:, 0] = -math.inf
        loss, _, dw = c.run()
        torch.cuda.synchronize()
        # the same logits in other tiles, or in other sums: within twice the bound of the one
        bound = ov.loss_and_gradients(c.hidden, c.weight[0][:128], c.ids, reduction="none", dtype="bf16")
        assert bool(((loss - want[0]).abs() <= 2 * bound[3]).all())
        assert bool(((dw[0][:128] - want[2]).abs() <= 2 * bound[5]).all()) and not bool(dw[0][128:].any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,temperature", [(1e8, 1.0), (1e10, 1.0), (3e12, 1.0), (1.0, 1e-7), (60.0, 1e-9)])
@pytest.mark.parametrize("T,top", [(60, 0), (60, 6), (200, 3)])
def test_logits_of_any_size(dtype, scale, temperature, T, top):
    """The exponent of a row's largest is 0, whatever rounding its logit takes on."""
    Case(T, 40, [500], dtype, top, seed=39, scale=scale, temperature=temperature).check()


@pytest.mark.parametrize("top", [0, 1, 6])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_target_far_ahead(dtype, top):
    """Logits near 1500 whose largest, the target's, leads by more than 200: the others' exponentials, below 2^-288,
    are 0 in fp32, the sum around the largest 1, and loss and gradients 0 to the last bit."""
    torch = torch_mod()
    for T in (50, 200):
        c = Case(T, 40, [700], dtype, top, seed=40, reduction="sum")
        c.weight[0].mul_(1e-3)
        c.weight[0][:, 0] = 120 + torch.rand(700, generator=torch.Generator(device="cuda").manual_seed(41), device="cuda")
        c.hidden[:, 0] = 9 + torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(42), device="cuda")
        c.weight[0][321, 0] = 151.3
        c.ids.fill_(-1 if top else 321)
        if top:
            c.ids[:, 0] = 321
        loss, dh, dw = c.run()
        assert float(c.run(False)) == 0 and float(loss) == 0 and not bool(dh.any()) and not bool(dw[0].any())


@pytest.mark.parametrize("T", [5, 50, 200])
@pytest.mark.parametrize("top", [0, 6])
def test_close_logits_far_from_zero(T, top):
    """Logits 1472 + v % 8, 1487 at v = 77, that every sum holds exactly (64 times 23 + v % 8 / 64, all other products
    0): the roundings that are left are the softmax's own, of differences of at most 15. An exponential's argument (two
    roundings of at most 22 in units of log 2), itself, and its place in a sum (a lane's 32, its neighbours', 3 tiles:
    under 48 levels) are off by (2 * 22 + 4 + 48) U of p, a teacher's probability by as much, D by 8 U more; dW = 64
    sum D adds 6 T + 64 roundings (six products, five of them zeros), dh of 300 terms 6 * 300 + 64."""
    torch = torch_mod()
    c = Case(T, 40, [300], "fp32", top, seed=43, reduction="sum", temperature=1.0)
    c.hidden.zero_()
    c.hidden[:, 5] = 64
    c.weight[0].zero_()
    c.weight[0][:, 5] = 23 + torch.arange(300, device="cuda") % 8 / 64
    c.weight[0][77, 5] = 23 + 15 / 64
    if top:
        c.ids[:, 0] = 77
    else:
        c.ids[:] = 77
    loss, dh, dw = c.run()
    want = c.want(False)
    W, h = c.weight[0].double(), c.hidden.double()
    p = torch.softmax(h @ W.t(), 1)
    ids = c.ids.reshape(T, -1)
    q = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), (ids >= 0).double())  # at least the target's or teacher's
    dD = 104 * ov.U * (p + q)
    assert abs(float(loss) - float(want[0])) <= T * 15 * 2 * 104 * ov.U
    within(dw[0], want[2], dD.t() @ h + (6 * T + 64) * ov.U * ((p + q).t() @ h) + 2.0 ** -120, "d_weight")
    within(dh, want[1], dD @ W + (6 * 300 + 64) * ov.U * ((p + q) @ W) + 2.0 ** -120, "d_hidden")


@pytest.mark.parametrize("top", [3, 6])
@pytest.mark.parametrize("T", [4, 200])
def test_a_teachers_logits_over_a_small_temperature(T, top):
    """Their quotients lie past the largest fp32 value, their differences' exponentials do not."""
    torch = torch_mod()
    c = Case(T, 40, [200], "fp32", top, seed=44, temperature=1e-37)
    c.hidden.zero_()
    c.ids = (torch.arange(T, device="cuda")[:, None] * 7 + torch.arange(top, device="cuda")) % 200
    c.logits[:] = 300 - 90.0 * torch.arange(top, device="cuda")
    c.logits[1, 0] = c.logits[1, 1]
    loss, dh, _ = c.check()
    assert math.isfinite(float(loss)) and bool(dh.any())


@pytest.mark.parametrize("T", [2, 200])
def test_a_weight_over_a_small_temperature(T):
    """A row's weight over the temperature may pass the largest fp32 value before it is divided by the rows."""
    torch = torch_mod()
    c = Case(T, 40, [200], "fp32", seed=45, temperature=1e-38, token_weights=torch.full((T,), 8.0, device="cuda"))
    c.hidden.zero_()
    for w in c.weight:
        w.mul_(1e-3)
    if T == 2:
        c.kw["token_weights"].fill_(4.0)
    loss, dh, dw = c.check()
    assert math.isfinite(float(loss)) and bool(dh.any()) and bool(torch.isfinite(dh).all())


def test_more_tokens_than_a_launch_has_workgroups_for():
    """2^26 rows and a few, 16 to a workgroup of 1024 that joins: 2^32 work-items, one more than a launch may have.
    Products of small whole numbers are exact, so a loss is off by its softmax and its own operations only."""
    torch = torch_mod()
    T, H = (1 << 26) + 3, 8
    g = torch.Generator(device="cuda").manual_seed(48)
    h = torch.randint(-2, 3, (T, H), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    w = torch.randint(-2, 3, (2, H), generator=g, device="cuda").bfloat16()
    y = torch.randint(0, 2, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[::5] = -100
    each, total = lib().vocab_loss(h, w, y, "none"), lib().vocab_loss(h, w, y, "sum")
    sums = [0.0, 0.0]
    for r in torch.arange(T, device="cuda").split(1 << 24):
        z = h[r].double() @ w.double().t()
        lse = torch.logsumexp(z, 1)
        kept = y[r] >= 0
        zt = z.gather(1, y[r].long().clamp(min=0)[:, None])[:, 0]
        want = torch.where(kept, lse - zt, torch.zeros_like(lse))
        bound = torch.where(kept, (280 + 24 * (lse.abs() + zt.abs())) * ov.U, torch.zeros_like(lse))
        within(each[r], want, bound, "loss")
        sums[0] += float(want.sum())
        sums[1] += float(bound.sum())
    assert abs(float(total) - sums[0]) <= sums[1] + ov.U * abs(sums[0])


@pytest.mark.parametrize("limit", [1, 3, None])
@pytest.mark.parametrize("T,V,dtype,top", [(40, [300], "fp32", 0), (1000, [3000, 500], "bf16", 6), (5000, [700], "bf16", 0), (3300, [1 << 17], "fp32", 3)])
def test_the_loss_is_the_sum_of_its_rows(T, V, dtype, top, limit):
    """Whatever workgroups a call has, one chunk or two: the rows' own losses summed in 64 bits, and rounded."""
    torch = torch_mod()
    A = lib()
    c = Case(T, 24, V, dtype, top, seed=49, left_out=0.05, weights=True)
    prev = A.ar_set_launch_blocks(limit) if limit and T * sum(V) < 1 << 23 else None
    try:
        for turn in range(3):
            c.hidden.neg_()
            each, total, mean, with_grad = c.run(False, reduction="none"), c.run(False, reduction="sum"), c.run(False), c.run()[0]
            count = int((c.ids.reshape(T, -1) >= 0).any(1).sum())
            for got, want in ((total, each.double().sum()), (mean, each.double().sum() / count)):
                assert abs(float(got) - float(want)) <= ov.U * abs(float(want)) + T * 2.0 ** -52 * float(each.double().abs().sum())
            assert torch.equal(mean, with_grad)
    finally:
        if prev is not None:
            A.ar_set_launch_blocks(prev)


def exact_products(T, V, H, gain=1024.0):
    """fp32 inputs whose every sum has one product that is not 0: hidden row t is x_t at column t and 0 elsewhere, the
    logit at id a_t leads by hundreds, so that D is w_t at a_t and -w_t at y_t and 0 elsewhere, all of full 24 bits."""
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(46)
    x, w = 1 + torch.rand(T, generator=g, device="cuda"), 1 + torch.rand(T, generator=g, device="cuda")
    hidden = torch.zeros(T, H, device="cuda")
    t = torch.arange(T, device="cuda")
    hidden[t, t] = x
    weight = torch.rand(V, H, generator=g, device="cuda") + 0.5
    order = torch.randperm(V, generator=g, device="cuda")
    a, y = order[:T], order[T: 2 * T]
    weight[a, t] = gain * (1 + torch.rand(T, generator=g, device="cuda"))
    return hidden, weight, a, y, w


# rows, vocabulary: few rows' products, middle and large tiles
@pytest.mark.parametrize("T,V", [(12, 600), (60, 600), (200, 1000), (200, 50000)])
def test_fp32_products_keep_their_bits(T, V):
    """A product of two 24-bit values from three bf16 terms each: the parts left out are below 2^-25 of it (x1 y2, x2 y1
    and smaller: a second term is at most 2^-9 of the first's value, a third 2^-17), the six that are kept are exact in
    fp32 and their sum is rounded five times: (6 + 2) U of the product. Losing any of the six shows (the CPU tests
    say so). A loss is the difference of two, scaled twice: 3 U more of each, and of itself."""
    torch = torch_mod()
    H = 264
    hidden, weight, a, y, w = exact_products(T, V, H)
    loss, dh, dw = lib().vocab_loss_grad(hidden, weight, y, "none", token_weights=w)
    t = torch.arange(T, device="cuda")
    W, x, c = weight.double(), hidden.double()[t, t], w.double()
    za, zy = x * W[a, t], x * W[y, t]
    within(loss, c * (za - zy), 12 * ov.U * c * (za + zy), "loss")
    # two products a sum, and the sum's rounding
    within(dh, c[:, None] * (W[a] - W[y]), 10 * ov.U * c[:, None] * (W[a] + W[y]), "d_hidden")
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    want[a, t] = c * x
    want[y, t] = -c * x
    within(dw, want, 9 * ov.U * want.abs(), "d_weight")


def by_rows(c, rows, count):
    """The oracle's losses, gradients and bounds from `rows` rows at a time; c.kw's reduction is "none" or "sum", or "mean"
    of `count` rows."""
    torch = torch_mod()
    T = len(c.ids)
    kw = dict(c.kw)
    share = 1.0 / count if kw.get("reduction", "mean") == "mean" else 1.0
    weights = kw.pop("token_weights", torch.ones(T, device="cuda")).double() * share
    kw["reduction"] = "none"
    W = torch.cat(c.weight)
    each, dh, dw = [], [], 0
    beach, bh, bw = [], [], 0
    for r in torch.arange(T, device="cuda").split(rows):
        out = ov.loss_and_gradients(c.hidden[r], W, c.ids[r], None if c.logits is None else c.logits[r], dtype=c.dtype,
                                    **dict(kw, token_weights=weights[r]))
        each.append(out[0]), dh.append(out[1]), beach.append(out[3]), bh.append(out[4])
        dw, bw = dw + out[2], bw + out[5]
    return torch.cat(each), torch.cat(dh), dw, torch.cat(beach), torch.cat(bh), bw


# more than one chunk of 4 GiB: fp32 of 131072 ids takes some 3000 rows at a time, of 2^20 ids 256, bf16 of 2^20 1792. In one
# the last chunk's rows are all left out.
@pytest.mark.parametrize("dtype,T,V,top,kw", [
    ("fp32", 3400, [130072, 1000], 0, {}), ("fp32", 6500, [130072, 1000], 3, dict(weights=True)),
    ("fp32", 4500, [130072, 1000], 8, dict(weights=True, temperature=1.5)),
    ("fp32", 600, [1 << 19, 1 << 19], 6, dict(reduction="none")), ("fp32", 1100, [1 << 20], 2, dict(reduction="sum", left_out=0.6)),
    ("bf16", 2300, [1 << 20], 9, dict(reduction="none", left_out=0.05)), ("bf16", 2000, [1 << 19, 1 << 19], 4, dict(weights=True, left_out=0.02))])
def test_lists_weights_and_means_in_chunks(dtype, T, V, top, kw):
    torch = torch_mod()
    c = Case(T, 20, V, dtype, top, seed=47, **kw)
    loss, dh, dw = c.run()
    alone = c.run(False)
    count = int((c.ids.reshape(T, -1) >= 0).any(1).sum())
    # a chunk's sums have no more terms than the oracle's blocks, but for bf16, whose 1792 roundings of |D| |h| are
    # 1792 * 2^-24 * 2^8 of what D's own rounding gives
    each, want_h, want_w, beach, bh, bw = by_rows(c, 3300 if sum(V) < 1 << 20 else 512, count)
    if dtype == "bf16":
        bw = 1.03 * bw
    if c.kw.get("reduction", "mean") == "none":
        within(loss, each, beach, "loss")
        assert torch.equal(loss, alone)
    else:
        within(loss, each.sum(), beach.sum() + 4 * ov.U * each.sum().abs(), "loss")
        within(alone, each.sum(), beach.sum() + 4 * ov.U * each.sum().abs(), "loss alone")
    within(dh, want_h, bh, "d_hidden")
    within(torch.cat(dw), want_w, bw, "d_weight")


@pytest.mark.parametrize("T,H,V", [(13, 40, 300), (48, 64, 1000), (48, 61, 1000), (100, 200, 5000), (700, 72, 30000)])
@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_means_factor_is_not_rounded_into_d(T, H, V, top, dtype):
    """N times a mean's gradients are the sum's, but for the rounding of each result (in fp32 the factor's own and its
    product's as well): 1 / N, the same in every row, may not be rounded into what the products multiply."""
    c = Case(T, H, [V], dtype, top, seed=50)
    _, dh, dw = c.run()
    _, sh, sw = c.run(reduction="sum")
    n = int((c.ids.reshape(T, -1) >= 0).any(1).sum())
    assert n & (n - 1)
    u = {"bf16": 2 * ov.U_BF16 + 4 * ov.U, "fp32": 6 * ov.U}[dtype] * 1.01
    for mean, total in ((dh, sh), (dw[0], sw[0])):
        within(mean * 1.0, total.double() / n, u * total.double().abs() / n + 2.0 ** -120, "a mean's gradient")


@pytest.mark.parametrize("T,H,V", [(1, 64, [300]), (3, 256, [5000, 37]), (16, 61, [1000]), (17, 128, [20000]), (48, 64, [700, 300]),
                                   (64, 200, [3000]), (64, 33, [257]), (50, 2048, [9000])])
@pytest.mark.parametrize("top", [0, 3, 8])
def test_few_rows_gradients_in_bf16_keep_two_terms_of_d(T, H, V, top):
    """Up to 64 rows D is the sum of two bf16 values: off by 2^-16 of it where one would be by 2^-8, which few terms of a
    result do not even out."""
    torch = torch_mod()
    c = Case(T, H, V, "bf16", top, seed=51, weights=T > 3, left_out=0.1 if T > 3 else 0.0, temperature=0.7)
    loss, dh, dw = c.run()
    want = c.want(d_terms=2)
    within(loss, want[0], want[3], "loss")
    within(dh, want[1], want[4], "d_hidden")
    within(torch.cat(dw), want[2], want[5], "d_weight")


@pytest.mark.parametrize("limit", [1, 3])
def test_launch_limit_of_few_rows(limit):
    """Two terms of D, in the tiles that load W as it is and in those that bring it in order."""
    A = lib()
    cases = [Case(T, H, [300, 30], "bf16", top=top, seed=52, left_out=0.2) for T, H, top in ((20, 64, 0), (50, 64, 6), (50, 61, 3), (9, 33, 0))]
    prev = A.ar_set_launch_blocks(limit)
    try:
        for c in cases:
            c.check()
    finally:
        A.ar_set_launch_blocks(prev)
