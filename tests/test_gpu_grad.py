"""Gradient norms and clipping on the GPU against their definition in 64 bits (oracle/grad.py).

Tolerances, with u = 2^-24, the largest relative error of a rounding to fp32, and 2^-8 that of one
to bf16:
* a norm is an fp64 value (its own error, below 2^-50 for these sizes, counted as SLACK) rounded to
  fp32 once: u;
* a scaled element is the product of two fp32 values, the factor itself rounded to fp32: 2 u,
  and 2^-8 more where it is stored in bf16. Results below the smallest normal value are off by half
  its last bit at most: 2^-150 in fp32, 2^-134 in bf16;
* the Allreduce's sums are held to the oracle's bits (rank order, fp32), so its results carry the same
  bounds.
"""
import math

import numpy as np
import pytest

import oracle
from oracle import grad as og
from synth import inputs
from gpu_util import from_device, to_device, torch_mod

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SLACK = 1 + 2.0 ** -40
TYPES = ("fp32", "bf16")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    torch.cuda.set_device(0)


def lib():
    import allreduce_schedule_algorithms_amd as A
    return A


def host_bits(t):
    torch = torch_mod()
    t = t.detach().contiguous()
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def values(n, dtype, seed, sigma=1.0):
    v = inputs.normal_fp32(1, n, seed, sigma)[0]
    return inputs.fp32_to_bf16_bits(v) if dtype == "bf16" else v


def on_gpu(bits, offset=0):
    """The buffer on the GPU, `offset` elements into an allocation with margins of a known pattern."""
    torch = torch_mod()
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16) if bits.dtype == np.uint16 else torch.from_numpy(bits)
    big = torch.full((bits.size + offset + 16,), 7.0, dtype=t.dtype, device="cuda")
    view = big[offset: offset + bits.size]
    view.copy_(t.cuda())
    return view, big


def margins_kept(big, offset, n):
    return bool((big[:offset] == 7).all()) and bool((big[offset + n:] == 7).all())


def types_of(kind, count):
    return [kind if kind in TYPES else TYPES[i % 2] for i in range(count)]


def close(got, want, rel, tiny=0.0):
    """Elementwise: |got - want| <= rel |want| + tiny where want is finite, and the same value where not."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    fin = np.isfinite(want)
    if not np.array_equal(np.isnan(got), np.isnan(want)):
        return False
    inf = np.isinf(want)
    if not np.array_equal(got[inf], want[inf]):
        return False
    return bool(np.all(np.abs(got[fin] - want[fin]) <= (rel * np.abs(want[fin]) + tiny) * SLACK))


def fits(got_bits, want, bf16):
    """A scaled result against its exact value."""
    rel = (1 + 2 * U + U * U) * (1 + 2.0 ** -8) - 1 if bf16 else 2 * U + U * U
    return close(og.widen(got_bits), want, rel, 2.0 ** -134 if bf16 else 2.0 ** -150)


# sizes around a vector, a workgroup's round, a work item and its end; lists of more tensors than a
# launch's table holds; empty tensors in front, between and behind
LISTS = {
    "none": [0], "one": [1], "two": [2, 0], "vector": [3, 4, 5, 7, 8, 9, 15, 16, 17],
    "item": [2047, 2048, 2049, 4095, 4097, 1], "empty": [0, 0, 5, 0, 2048, 0, 0, 3, 0],
    "table": [1 + i % 11 for i in range(129)], "long": [(i * 37) % 301 for i in range(1000)],
    "large": [1_000_003, 17, 300_007, 2_500_000],
}


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("types", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("name", list(LISTS))
def test_norms(name, types, kind):
    A = lib()
    sizes = LISTS[name]
    host = [values(n, d, 100 + i, 10.0 ** (i % 5 - 2)) for i, (n, d) in enumerate(zip(sizes, types_of(types, len(sizes))))]
    want, each = og.norms(host, kind)
    first = None
    for shift in (0, 1, 5):
        dev = [on_gpu(b, shift and (i + shift) % 8) for i, b in enumerate(host)]
        total, own = A.grad_norm([v for v, _ in dev], norm=kind, per_tensor=True)
        alone = A.grad_norm([v for v, _ in dev], norm=kind)
        assert total.shape == () and own.shape == (len(sizes),)
        assert close(float(total), want, U) and close(own.cpu().numpy(), each, U)
        # the cut goes by sizes alone: the same bits at every address, on every run
        bits = (total.cpu().numpy().tobytes(), own.cpu().numpy().tobytes())
        first = first or bits
        assert bits == first and alone.cpu().numpy().tobytes() == bits[0]


def test_one_tensor_is_a_list_of_one():
    A, torch = lib(), torch_mod()
    t = torch.full((30, 30), 2.0, device="cuda")
    o = torch.empty_like(t, dtype=torch.bfloat16)
    total, own = A.grad_norm(t, per_tensor=True)
    assert float(total) == 60 and own.shape == (1,)
    assert float(A.grad_clip(t, 30.0, eps=0.0, out=o)) == 60 and bool((o == 1).all()) and bool((t == 2).all())


def test_no_tensors():
    A = lib()
    total, own = A.grad_norm([], per_tensor=True)
    assert float(total) == 0 and own.numel() == 0
    assert float(A.grad_clip([], 1.0)) == 0


SPECIAL = {
    "zeros": [0.0, -0.0, 0.0], "overflow": [3e38, -3e38, 1.0], "squares_overflow": [1e30, 2e30, -3e30],
    "vanish": [1e-40, -2e-40, 1e-45], "squares_vanish": [1e-30, 2e-30], "inf": [1.0, math.inf, 2.0], "neg_inf": [-math.inf, 1.0],
    "nan": [1.0, math.nan, 2.0], "nan_and_inf": [math.inf, math.nan, -math.inf], "neg_nan": [-math.nan, 5.0],
    "wide": [1e30, 1e-30, 1.0],
}


@pytest.mark.parametrize("name", list(SPECIAL))
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(name, kind, dtype):
    A, torch = lib(), torch_mod()
    v = np.zeros(4099, np.float32)
    v[[0, 2050, 4098][: len(SPECIAL[name])]] = np.float32(SPECIAL[name])
    t = torch.from_numpy(v).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    host = host_bits(t)
    want, _ = og.norms([host], kind)
    with np.errstate(over="ignore"):
        shown = float(np.float32(want))  # a norm past fp32's range is its infinity
    got = A.grad_norm([t.cuda()], norm=kind)
    assert close(float(got), shown, U, 2.0 ** -150)
    # the factor comes from the norm itself, not from its fp32 value
    f = og.factor(want, 1.0, 1e-6)
    with np.errstate(invalid="ignore"):
        exact = og.widen(host) * f
    d = t.cuda()
    A.grad_clip([d], 1.0, norm=kind)
    assert fits(host_bits(d), exact, dtype == "bf16")


@pytest.mark.parametrize("out", ["in_place", "fp32", "bf16"])
@pytest.mark.parametrize("types", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("name", list(LISTS))
def test_clip(name, types, out):
    A, torch = lib(), torch_mod()
    sizes = LISTS[name]
    src = types_of(types, len(sizes))
    host = [values(n, d, 300 + i, 10.0 ** (i % 4 - 2)) for i, (n, d) in enumerate(zip(sizes, src))]
    for kind, shift in (("l2", 0), ("max", 3)):
        norm, _ = og.norms(host, kind)
        for max_norm in (norm / 3, norm * 2 + 1):
            f = og.factor(norm, max_norm, 1e-6)
            dev = [on_gpu(b, shift and (i + shift) % 8) for i, b in enumerate(host)]
            if out == "in_place":
                outs, dst, places = None, src, dev
            else:
                dst = [out] * len(sizes)
                places = [on_gpu(np.zeros(n, np.float32 if out == "fp32" else np.uint16), (2 * i + shift) % 8 if shift else 0)
                          for i, n in enumerate(sizes)]
                outs = [v for v, _ in places]
            got = A.grad_clip([v for v, _ in dev], max_norm, norm=kind, out=outs)
            assert close(float(got), norm, U)
            for i, n in enumerate(sizes):
                view, big = places[i]
                bits = host_bits(view)
                assert fits(bits, og.widen(host[i]) * f, dst[i] == "bf16"), (i, n, kind, max_norm)
                if f == 1.0 and dst[i] == src[i]:
                    assert np.array_equal(bits.view(np.uint8), host[i].view(np.uint8)), "a gradient within the limit keeps its bits"
                at = (view.data_ptr() - big.data_ptr()) // view.element_size()
                assert margins_kept(big, at, n)
                if out != "in_place":
                    assert np.array_equal(host_bits(dev[i][0]).view(np.uint8), host[i].view(np.uint8)), "inputs are left alone"


@pytest.mark.parametrize("max_norm,eps", [(0.0, 1e-6), (0.0, 0.0), (math.inf, 1e-6), (1e-30, 1e-6), (3.4e38, 0.0), (0.5, 0.25),
                                          (1e-38, 0.0), (1e-45, 0.0)])
def test_limits(max_norm, eps):
    A = lib()
    for dtype in TYPES:
        for sigma in (1.0, 1e37):
            host = values(5000, dtype, 5, sigma)
            norm, _ = og.norms([host], "l2")
            view, _ = on_gpu(host)
            A.grad_clip([view], max_norm, eps=eps)
            assert fits(host_bits(view), og.widen(host) * og.factor(norm, max_norm, eps), dtype == "bf16")
    z, _ = on_gpu(np.zeros(100, np.float32))
    A.grad_clip([z], max_norm, eps=eps)
    assert not host_bits(z).any()


@pytest.mark.parametrize("known", [0.25, 1.0, 7.5, 0.0, math.inf, math.nan])
def test_clip_by_a_known_norm(known):
    A, torch = lib(), torch_mod()
    host = [values(n, d, n) for n, d in ((5000, "fp32"), (3001, "bf16"), (0, "fp32"))]
    f = og.factor(float(np.float32(known)), 1.0, 1e-6)
    dev = [on_gpu(b, 1) for b in host]
    k = torch.tensor(known, dtype=torch.float32, device="cuda")
    assert A.grad_clip([v for v, _ in dev], 1.0, total_norm=k) is k
    for b, (v, _) in zip(host, dev):
        with np.errstate(invalid="ignore"):
            assert fits(host_bits(v), og.widen(b) * f, b.dtype == np.uint16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value,max_norm", [(3e38, 1e-45), (1.7e38, 1e-45), (3.38e38, 3e-45), (3e38, 1e-38), (-2e38, 7e-45)])
def test_the_smallest_scales(value, max_norm, dtype):
    """One element past the limit becomes the limit, down to scales of 2^-277; the limit itself where that is a
    few steps of 2^-149, of which the factors' roundings are a small part."""
    A, torch = lib(), torch_mod()
    t = torch.tensor([0.0, value, -0.0], dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    for host in (host_bits(t), np.concatenate([host_bits(t)] + [np.zeros_like(host_bits(t))] * 20_000)):
        norm, _ = og.norms([host], "l2")
        f = og.factor(norm, max_norm, 0.0)
        out = torch.zeros(host.size, device="cuda")
        view, _ = on_gpu(host)
        A.grad_clip([view], max_norm, eps=0.0, out=[out])
        assert fits(host_bits(out), og.widen(host) * f, False)
        assert max_norm > 1e-40 or float(out[1]) == math.copysign(float(np.float32(max_norm)), value)
        A.grad_clip([view], max_norm, eps=0.0)
        assert fits(host_bits(view), og.widen(host) * f, dtype == "bf16")


@pytest.mark.parametrize("dtype", TYPES)
def test_an_infinity_by_a_known_norm_and_the_smallest_scale(dtype):
    A, torch = lib(), torch_mod()
    t = torch.tensor([math.inf, 1.0, -math.inf, math.nan, 3e38], dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    known = torch.tensor([3e38], device="cuda")
    for max_norm in (1e-45, 1e-30, 1.0):
        f = og.factor(float(known), max_norm, 1e-6)
        got, want = t.clone(), og.widen(host_bits(t)) * f
        A.grad_clip([got], max_norm, total_norm=known)
        assert fits(host_bits(got), want, dtype == "bf16")


# ---- the Allreduce that clips ----
def ranks_on_gpu(x, offset=0):
    """One view per rank, rank p `offset + p` elements (mod 8) into its allocation where offset is not 0."""
    return [on_gpu(np.ascontiguousarray(x[p]), offset and (offset + p) % 8) for p in range(x.shape[0])]


def check_allreduce_clip(hosts, op, kind, collective, max_of, offset=0, eps=1e-6, stream=None):
    """hosts: (P, n) bits of every bucket."""
    A, torch = lib(), torch_mod()
    bf16 = hosts[0].dtype == np.uint16
    norm = og.allreduce_clip(hosts, 1.0, eps, op, kind)[0]
    max_norm = max_of(norm)
    norm, f, want = og.allreduce_clip(hosts, max_norm, eps, op, kind)
    dev = [ranks_on_gpu(x, offset) for x in hosts]
    got = A.allreduce_clip([[v for v, _ in d] for d in dev], max_norm, op=op, norm=kind, eps=eps, collective=collective,
                           stream=stream)
    torch.cuda.synchronize()
    assert close(float(got), norm, U)
    for x, d, w in zip(hosts, dev, want):
        P, n = x.shape
        part = -(-n // P) if n else 0
        exactly = None
        if f == 1.0:
            c = og.combine(x, op)
            exactly = inputs.fp32_to_bf16_bits(c) if bf16 else c
        for p, (view, big) in enumerate(d):
            bits = host_bits(view)
            lo, hi = (0, n) if collective == "allreduce" else (min(p * part, n), min((p + 1) * part, n))
            assert fits(bits[lo:hi], w[lo:hi], bf16), (p, P, n, op, kind)
            if exactly is not None:
                assert np.array_equal(bits[lo:hi].view(np.uint8), exactly[lo:hi].view(np.uint8))
            for a, b in ((0, lo), (hi, n)):
                assert np.array_equal(bits[a:b].view(np.uint8), x[p, a:b].view(np.uint8)), "other parts are untouched"
            at = (view.data_ptr() - big.data_ptr()) // view.element_size()
            assert margins_kept(big, at, n)


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P", [1, 2, 3, 7, 8, 9, 24, 65, 256])
def test_allreduce_clip(P, dtype, collective):
    for n in (0, 1, 2, 5, 106, 1001, 4099) + ((70_001,) if P <= 24 else ()):
        x = inputs.make(dtype, P, n, seed=P * 31 + n)
        for op, kind, offset in (("sum", "l2", 0), ("avg", "max", 0), ("sum", "max", 1), ("avg", "l2", 3)):
            check_allreduce_clip([x], op, kind, collective, lambda N: N / 3, offset)
        check_allreduce_clip([x], "sum", "l2", collective, lambda N: 2 * N + 1, P % 2)


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P,sizes", [(3, [1, 0, 5000, 7, 2048, 0]), (8, [30_000, 106, 9]), (24, [100 + i for i in range(40)]),
                                     (200, [50, 3000, 1, 0, 7]), (256, [300, 300, 300])])
def test_allreduce_clip_buckets(P, sizes, dtype, collective):
    hosts = [inputs.make(dtype, P, n, seed=n + i) for i, n in enumerate(sizes)]
    for op, kind, offset in (("sum", "l2", 0), ("avg", "max", 5)):
        check_allreduce_clip(hosts, op, kind, collective, lambda N: N / 2, offset)


def test_allreduce_clip_each_bucket():
    A, torch = lib(), torch_mod()
    hosts = [inputs.make("bf16", 5, n, seed=n) for n in (0, 40, 9000)]
    dev = [[v for v, _ in ranks_on_gpu(x)] for x in hosts]
    total, each = torch.empty((), device="cuda"), torch.empty(3, device="cuda")
    A.ar_allreduce_clip([t for d in dev for t in d], [0, 40, 9000], 5, "bf16", "sum", "allreduce",
                        A.make_clip("l2", 1.0, total=total, each=each), torch.cuda.current_stream())
    want = [og.norm_of(og.combine(x, "sum").astype(np.float64), "l2") for x in hosts]
    assert close(each.cpu().numpy(), want, U)


def test_allreduce_clip_within_the_limit_is_the_direct_allreduce():
    A, torch = lib(), torch_mod()
    for dtype in TYPES:
        for op in ("sum", "avg"):
            x = inputs.make(dtype, 7, 12_345, seed=4)
            a, _ = to_device(x, dtype)
            b, _ = to_device(x, dtype)
            A.allreduce(a, algo="direct", op=op)
            A.allreduce_clip(b, math.inf, op=op)
            assert np.array_equal(from_device(a, dtype).view(np.uint8), from_device(b, dtype).view(np.uint8))


@pytest.mark.parametrize("name", ["overflow", "inf", "nan", "nan_and_inf", "vanish", "zeros"])
@pytest.mark.parametrize("dtype", TYPES)
def test_allreduce_clip_special_values(name, dtype):
    torch = torch_mod()
    x = np.zeros((3, 4099), np.float32)
    for p, v in enumerate(SPECIAL[name]):
        x[p, [0, 2050, 4098][p]] = v
    t = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    host = host_bits(t)
    with np.errstate(invalid="ignore", over="ignore"):
        norm, f, want = og.allreduce_clip([host], 1.0, 1e-6, "sum", "l2")
        A = lib()
        dev = [v for v, _ in ranks_on_gpu(host)]
        got = A.allreduce_clip(dev, 1.0)
        assert close(float(got), float(np.float32(norm)), U, 2.0 ** -150)
        for v in dev:
            assert fits(host_bits(v), want[0], dtype == "bf16")


# ---- together ----
@pytest.mark.parametrize("dtype", TYPES)
def test_a_training_step(dtype):
    """Reduce, measure, clip into fp32 gradients: the separate calls against the one call and the oracle."""
    A, torch = lib(), torch_mod()
    P, sizes = 4, [5000, 333, 70_001]
    hosts = [inputs.make(dtype, P, n, seed=n) for n in sizes]
    norm, f, want = og.allreduce_clip(hosts, 2.0, 1e-6, "avg", "l2")
    one = [[v for v, _ in ranks_on_gpu(x)] for x in hosts]
    fused = A.allreduce_clip(one, 2.0, op="avg")
    apart = [[v for v, _ in ranks_on_gpu(x)] for x in hosts]
    for b in apart:
        A.allreduce(b, algo="direct", op="avg")
    grads = [b[0] for b in apart]
    main = [torch.empty(n, device="cuda") for n in sizes]
    measured, each = A.grad_norm(grads, per_tensor=True)
    clipped = A.grad_clip(grads, 2.0, out=main, total_norm=measured)
    again = A.grad_clip(grads, 2.0)
    assert torch.equal(again, measured) and clipped is measured
    # separate calls see the reduced values after their rounding to dtype
    rounding = 2.0 ** -8 if dtype == "bf16" else U
    assert close(float(fused), norm, U) and close(float(measured), norm, U + rounding)
    assert close(float((each.double() ** 2).sum().sqrt()), float(measured), 4 * U)
    for b, g, m, w in zip(one, grads, main, want):
        assert close(m.cpu().numpy(), w, 2 * rounding + 6 * U)
        assert close(og.widen(host_bits(g)), w, 3 * rounding + 6 * U)
        for v in b:
            assert fits(host_bits(v), w, dtype == "bf16")


# ---- streams, graphs, workspaces ----
def test_another_stream():
    A, torch = lib(), torch_mod()
    s = torch.cuda.Stream()
    host = [values(n, "bf16", n) for n in (100_003, 5000)]
    norm, _ = og.norms(host, "l2")
    dev = [on_gpu(b)[0] for b in host]
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = A.grad_norm(dev, stream=stream)
        s.synchronize()
        assert close(float(got), norm, U)
    with torch.cuda.stream(s):
        got = A.grad_clip(dev, norm / 2)
    s.synchronize()
    assert close(float(got), norm, U)
    for b, v in zip(host, dev):
        assert fits(host_bits(v), og.widen(b) * og.factor(norm, norm / 2, 1e-6), True)
    check_allreduce_clip([inputs.make("fp32", 4, 5001, seed=1)], "sum", "l2", "allreduce", lambda N: N / 2, stream=s)


def test_two_streams_at_once():
    A, torch = lib(), torch_mod()
    streams = [torch.cuda.Stream() for _ in range(2)]
    hosts = [[values(n, "fp32", 10 * k + n % 7, 1.0 + k) for n in (400_001, 2_000_003, 77)] for k in range(2)]
    dev = [[on_gpu(b)[0] for b in h] for h in hosts]
    want = [og.norms(h, "l2")[0] for h in hosts]
    tables = [A.marshal_grads([(t.data_ptr(), 0, t.numel(), "fp32", "fp32") for t in d]) for d in dev]
    totals = torch.empty(2, 20, device="cuda")
    torch.cuda.synchronize()
    for r in range(20):  # the library's own workspace: one for each stream
        for k in range(2):
            A.ar_grad_norm(tables[k], A.make_clip(total=totals[k, r].data_ptr()), streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert close(totals[k].cpu().numpy(), np.full(20, want[k]), U)


def test_threads_on_one_stream():
    import threading
    A, torch = lib(), torch_mod()
    hosts = [[values(n, "fp32", 10 * k + n % 7, 1.0 + k) for n in (300_001, 1_000_003)] for k in range(3)]
    dev = [[on_gpu(b)[0] for b in h] for h in hosts]
    want = [og.norms(h, "l2")[0] for h in hosts]
    tables = [A.marshal_grads([(t.data_ptr(), 0, t.numel(), "fp32", "fp32") for t in d]) for d in dev]
    totals = torch.empty(3, 50, device="cuda")
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            for r in range(50):
                A.ar_grad_norm(tables[k], A.make_clip(total=totals[k, r].data_ptr()), stream)
        except Exception as e:  # shown by the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not failed
    for k in range(3):
        assert close(totals[k].cpu().numpy(), np.full(50, want[k]), U)


def test_graphs():
    """Two captured graphs, replayed in turn with eager calls between them, each replay against the eager result."""
    A, torch = lib(), torch_mod()
    sizes = (200_003, 17, 4096)
    pristine = [torch.randn(n, device="cuda") for n in sizes]
    grads = [t.clone() for t in pristine]
    main = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
    rows = torch.randn(5, 30_001, device="cuda")
    ranks = [t.clone() for t in rows]
    A.grad_clip(grads, 3.0, out=main)
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        na = A.grad_clip(grads, 3.0, out=main)
    with torch.cuda.graph(b):
        nb = A.allreduce_clip(ranks, 2.0)
    for k in range(4):
        fresh = [t * (k + 1) for t in pristine]
        [g.copy_(f) for g, f in zip(grads, fresh)]
        [r.copy_(x * (k + 1)) for r, x in zip(ranks, rows)]
        eager_main = [torch.empty_like(m) for m in main]
        ea = A.grad_clip(fresh, 3.0, out=eager_main)
        eager_ranks = [x * (k + 1) for x in rows]
        eb = A.allreduce_clip(eager_ranks, 2.0)
        torch.cuda.synchronize()
        a.replay()
        b.replay()
        other = A.grad_norm(fresh[:2])
        torch.cuda.synchronize()
        assert torch.equal(na, ea) and torch.equal(nb, eb)
        assert all(torch.equal(x, y) for x, y in zip(main, eager_main))
        assert all(torch.equal(x, y) for x, y in zip(ranks, eager_ranks))
        assert close(float(other), og.norms([host_bits(t) for t in fresh[:2]], "l2")[0], U)


def test_capture_needs_a_workspace():
    A, torch = lib(), torch_mod()
    n = 1_000_000
    t = torch.ones(n, device="cuda")
    total = torch.zeros((), device="cuda")
    table = A.marshal_grads([(t.data_ptr(), 0, n, "fp32", "fp32")])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        total.add_(1)
        s = torch.cuda.current_stream()
        for call in (lambda: A.ar_grad_norm(table, A.make_clip(total=total), s),
                     lambda: A.ar_grad_clip(table, A.make_clip(max_norm=1.0), s),
                     lambda: A.ar_allreduce_clip([t], [n], 1, "fp32", "sum", "allreduce", A.make_clip(max_norm=1.0), s)):
            with pytest.raises(A.ArError) as e:
                call()
            assert e.value.status == A.Status.AR_UNSUPPORTED
    g.replay()
    torch.cuda.synchronize()
    assert float(total) == 1 and bool((t == 1).all())


def test_workspaces():
    A, torch = lib(), torch_mod()
    host = [values(n, "bf16", n) for n in (500_001, 300)]
    norm, _ = og.norms(host, "l2")
    dev = [on_gpu(b)[0] for b in host]
    table = A.marshal_grads([(t.data_ptr(), 0, t.numel(), "bf16", "bf16") for t in dev])
    need = A.ar_grad_workspace_bytes(table, A.make_clip())
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    total = torch.zeros((), device="cuda")
    s = torch.cuda.current_stream()
    with pytest.raises(A.ArError) as e:
        A.ar_grad_norm(table, A.make_clip(total=total, workspace=ws, workspace_bytes=need - 1), s)
    assert e.value.status == A.Status.AR_WORKSPACE_TOO_SMALL
    A.ar_grad_norm(table, A.make_clip(total=total, workspace=ws, workspace_bytes=need), s)
    assert close(float(total), norm, U) and bool((ws[need:] == 255).all())
    assert close(float(A.grad_norm(dev, workspace=ws)), norm, U)
    x = inputs.make("bf16", 6, 10_001, seed=2)
    ranks = [v for v, _ in ranks_on_gpu(x)]
    args = ([10_001], 6, "bf16", "sum", "reduce_scatter")
    need = A.ar_allreduce_clip_workspace_bytes(*args, A.make_clip(max_norm=1.0))
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    A.ar_allreduce_clip(ranks, *args, A.make_clip(max_norm=1.0, workspace=ws, workspace_bytes=need), s)
    torch.cuda.synchronize()
    want = og.allreduce_clip([x], 1.0, 1e-6, "sum", "l2")[2][0]
    part = -(-10_001 // 6)
    for p, v in enumerate(ranks):
        assert fits(host_bits(v)[p * part:(p + 1) * part], want[p * part:(p + 1) * part], True)
    assert bool((ws[need:] == 255).all())


def test_library_workspaces_are_counted_and_released():
    A, torch = lib(), torch_mod()
    t = torch.ones(1_000_000, device="cuda")
    table = A.marshal_grads([(t.data_ptr(), 0, t.numel(), "fp32", "fp32")])
    total = torch.zeros((), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = A.ar_cache_stats_get()
    A.ar_grad_norm(table, A.make_clip(total=total), s)
    after = A.ar_cache_stats_get()
    assert after["workspaces"] == before["workspaces"] + 1
    assert after["workspace_device_bytes"] > before["workspace_device_bytes"]
    s.synchronize()
    assert float(total) == 1000
    A.ar_release_cached()
    assert A.ar_cache_stats_get()["workspaces"] == 0
    A.ar_grad_norm(table, A.make_clip(total=total), s)
    s.synchronize()
    assert float(total) == 1000


def test_launch_limit_and_events():
    A, torch = lib(), torch_mod()
    host = [values(n, "fp32", n) for n in (100_003, 9000)]
    norm, _ = og.norms(host, "l2")
    old = A.ar_set_launch_blocks(3)
    try:
        dev = [on_gpu(b)[0] for b in host]
        assert close(float(A.grad_norm(dev)), norm, U)
        A.grad_clip(dev, norm / 2)
        for b, v in zip(host, dev):
            assert fits(host_bits(v), og.widen(b) * og.factor(norm, norm / 2, 1e-6), False)
        check_allreduce_clip([inputs.make("bf16", 5, 50_001, seed=3)], "sum", "l2", "allreduce", lambda N: N / 2)
    finally:
        A.ar_set_launch_blocks(old)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record(), stop.record()
    torch.cuda.synchronize()
    s = torch.cuda.current_stream()
    total = torch.zeros((), device="cuda")
    for records in ([(t.data_ptr(), 0, t.numel(), "fp32", "fp32") for t in dev], []):
        clip = A.make_clip(max_norm=1.0, total=total, start_event=start, stop_event=stop)
        A.ar_grad_clip(A.marshal_grads(records), clip, s)
        torch.cuda.synchronize()
        assert 0 <= start.elapsed_time(stop) < 1000


def test_offsets_past_32_bits():
    """More than 2^32 elements in one tensor and in one bucket, values placed at both ends."""
    A, torch = lib(), torch_mod()
    n = (1 << 32) + 12_345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[0], t[1 << 31], t[1 << 32], t[-1] = 1.0, 2.0, 4.0, 10.0
    assert float(A.grad_norm([t])) == 11.0
    assert float(A.grad_norm([t], norm="max")) == 10.0
    assert float(A.grad_clip([t], 5.5, eps=0.0)) == 11.0
    assert [float(v) for v in (t[0], t[1 << 31], t[1 << 32], t[-1])] == [0.5, 1.0, 2.0, 5.0]
    other = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    other[-1] = 5.0
    # sums 0.5, 1, 2, 10: norm sqrt(105.25)
    got = A.allreduce_clip([t, other], 1e9)
    assert close(float(got), math.sqrt(105.25), U)
    for b in (t, other):
        assert [float(v) for v in (b[0], b[1 << 31], b[1 << 32], b[-1])] == [0.5, 1.0, 2.0, 10.0]
        assert int((b != 0).sum()) == 4


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P", [1, 2, 3, 4, 5, 6, 7, 8, 9, 24, 40])
def test_allreduce_clip_long(P, dtype, collective):
    # past the sizes that are cut finer: items of 2048 elements and more, every batch of ranks
    n = 300_011 if P <= 9 else 262_147
    x = inputs.make(dtype, P, n, seed=P)
    check_allreduce_clip([x], "avg" if P % 2 else "sum", "l2" if P % 3 else "max", collective, lambda N: N / 3, P % 2 * 3)


@pytest.mark.parametrize("limit", [1, 3, 16_777_215])
def test_own_norms_under_a_launch_limit(limit):
    A, torch = lib(), torch_mod()
    sizes = [(i * 977) % 5000 for i in range(300)]
    host = [values(n, "fp32" if i % 3 else "bf16", i) for i, n in enumerate(sizes)]
    want, each = og.norms(host, "l2")
    dev = [on_gpu(b, i % 3)[0] for i, b in enumerate(host)]
    hosts = [inputs.make("bf16", 5, n, seed=n) for n in (0, 40_000, 9000, 300_000, 7)]
    ranks = [v for x in hosts for v, _ in ranks_on_gpu(x)]
    sums = [og.combine(x, "avg").astype(np.float64) for x in hosts]
    total, own = torch.empty((), device="cuda"), torch.empty(len(hosts), device="cuda")
    old = A.ar_set_launch_blocks(limit)
    try:
        got, norms = A.grad_norm(dev, per_tensor=True)
        A.ar_allreduce_clip(ranks, [x.shape[1] for x in hosts], 5, "bf16", "avg", "allreduce",
                            A.make_clip("l2", 1.0, total=total, each=own), torch.cuda.current_stream())
        torch.cuda.synchronize()
    finally:
        A.ar_set_launch_blocks(old)
    assert close(float(got), want, U) and close(norms.cpu().numpy(), each, U)
    assert close(own.cpu().numpy(), [og.norm_of(s, "l2") for s in sums], U)
    norm = og.norm_of(np.array([og.norm_of(s, "l2") for s in sums]), "l2")
    assert close(float(total), norm, U)
    for k, (x, s) in enumerate(zip(hosts, sums)):
        for p in range(5):
            assert fits(host_bits(ranks[5 * k + p]), s * og.factor(norm, 1.0, 1e-6), True)


def test_known_norm_over_several_tables():
    A, torch = lib(), torch_mod()
    host = [values((i * 311) % 4000, TYPES[i % 2], i) for i in range(400)]
    dev = [on_gpu(b, i % 5)[0] for i, b in enumerate(host)]
    out = [torch.empty(b.size, dtype=torch.bfloat16 if i % 3 else torch.float32, device="cuda") for i, b in enumerate(host)]
    A.grad_clip(dev, 2.0, out=out, total_norm=torch.tensor([8.0], device="cuda"))
    for b, o in zip(host, out):
        assert fits(host_bits(o), og.widen(b) * og.factor(8.0, 2.0, 1e-6), o.dtype == torch.bfloat16)


def test_an_earlier_calls_error_is_not_taken_for_this_ones():
    import ctypes
    A, torch = lib(), torch_mod()
    hip = ctypes.CDLL("libamdhip64.so.7")
    t = torch.full((100,), 2.0, device="cuda")
    torch.cuda.synchronize()
    assert hip.hipSetDevice(1000) != 0  # leaves an error for whoever asks for the thread's last one
    table = A.marshal_grads([(t.data_ptr(), 0, 100, "fp32", "fp32")])
    total = t.new_empty(())
    A.ar_grad_norm(table, A.make_clip(total=total), torch.cuda.current_stream())
    hip.hipGetLastError()
    assert float(total) == 20.0


@pytest.mark.parametrize("sizes", [[100, 0, 3, 2000], [100_003, 0, 40_000, 7], [1 + i % 900 for i in range(200)]], ids=["small", "large", "tables"])
def test_clip_with_own_norms(sizes):
    A, torch = lib(), torch_mod()
    host = [values(n, TYPES[i % 2], i) for i, n in enumerate(sizes)]
    norm, each = og.norms(host, "l2")
    dev = [on_gpu(b)[0] for b in host]
    total, own = torch.empty((), device="cuda"), torch.full((len(sizes) + 1,), -1.0, device="cuda")
    table = A.marshal_grads([(t.data_ptr(), 0, t.numel(), d, d) for t, d in zip(dev, (TYPES[i % 2] for i in range(len(sizes))))])
    A.ar_grad_clip(table, A.make_clip("l2", norm / 4, total=total, each=own), torch.cuda.current_stream())
    assert close(float(total), norm, U) and close(own[:-1].cpu().numpy(), each, U) and float(own[-1]) == -1
    for b, v in zip(host, dev):
        assert fits(host_bits(v), og.widen(b) * og.factor(norm, norm / 4, 1e-6), b.dtype == np.uint16)


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
def test_own_norms_of_small_buckets(collective):
    A, torch = lib(), torch_mod()
    hosts = [inputs.make("fp32", 3, n, seed=n) for n in (5, 0, 130, 64)]
    dev = [v for x in hosts for v, _ in ranks_on_gpu(x)]
    total, own = torch.empty((), device="cuda"), torch.full((5,), -1.0, device="cuda")
    args = ([5, 0, 130, 64], 3, "fp32", "sum", collective)
    assert A.ar_allreduce_clip_workspace_bytes(*args, A.make_clip(max_norm=1.0, each=own)) == 0
    A.ar_allreduce_clip(dev, *args, A.make_clip("l2", 1.0, total=total, each=own), torch.cuda.current_stream())
    want = [og.norm_of(og.combine(x, "sum").astype(np.float64), "l2") for x in hosts]
    assert close(own[:-1].cpu().numpy(), want, U) and float(own[-1]) == -1
    assert close(float(total), og.norm_of(np.array(want), "l2"), U)


def test_clip_of_many_launches():
    """More partials than the scaling pass joins by itself: three tables and more, each with a full grid."""
    A, torch = lib(), torch_mod()
    sizes = [40_000 + i % 13 for i in range(600)]
    flat = torch.randn(sum(sizes), device="cuda")
    grads = list(flat.split(sizes))
    exact = flat.double()
    norm = float(exact.pow(2).sum().sqrt())
    got = A.grad_clip(grads, norm / 3)
    assert close(float(got), norm, U)
    want = exact * og.factor(norm, norm / 3, 1e-6)
    assert bool(((flat.double() - want).abs() <= 2 * U * SLACK * want.abs() + 2.0 ** -150).all())


def test_a_list_built_once():
    A, torch = lib(), torch_mod()
    host = [values(n, TYPES[i % 2], i) for i, n in enumerate((5000, 0, 77, 200_001))]
    norm, each = og.norms(host, "l2")
    dev = [on_gpu(b, i)[0] for i, b in enumerate(host)]
    out = [torch.empty(b.size, device="cuda") for b in host]
    table = A.grad_list(dev, out)
    with pytest.raises(A.ArError):
        A.grad_clip(table, 1.0, out=out)
    for _ in range(2):
        total, own = A.grad_norm(table, per_tensor=True)
        assert close(float(total), norm, U) and close(own.cpu().numpy(), each, U)
        assert close(float(A.grad_clip(table, norm / 2)), norm, U)
        for b, o in zip(host, out):
            assert fits(host_bits(o), og.widen(b) * og.factor(norm, norm / 2, 1e-6), False)
            o.zero_()
    dev[0].mul_(2)  # the list reads what its tensors hold
    host[0] = host_bits(dev[0])
    assert close(float(A.grad_norm(table)), og.norms(host, "l2")[0], U)


def test_the_per_thread_stream_needs_a_workspace():
    A, torch = lib(), torch_mod()
    per_thread = 2  # hipStreamPerThread
    t = torch.ones(1_000_000, device="cuda")
    total = torch.zeros((), device="cuda")
    table = A.grad_list([t])
    torch.cuda.synchronize()
    with pytest.raises(A.ArError) as e:
        A.ar_grad_norm(table, A.make_clip(total=total), per_thread)
    assert e.value.status == A.Status.AR_UNSUPPORTED
    ws = torch.empty(A.ar_grad_workspace_bytes(table, A.make_clip()), dtype=torch.uint8, device="cuda")
    A.ar_grad_norm(table, A.make_clip(total=total, workspace=ws, workspace_bytes=ws.numel()), per_thread)
    torch.cuda.synchronize()
    assert float(total) == 1000


@pytest.mark.parametrize("call", ["in_place", "out", "known", "list", "allreduce", "reduce_scatter", "buckets"])
def test_autograd_sees_what_is_written(call):
    """A tensor that autograd saved may not change before its backward pass: writing to it has to be seen."""
    A, torch = lib(), torch_mod()
    g, o = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda")
    other = torch.ones(5000, device="cuda")
    w = torch.ones(5000, device="cuda", requires_grad=True)
    known = torch.tensor(50.0, device="cuda")
    read, written = (g, o) if call == "out" else (other, g)
    kept, lost = (w * read).sum(), (w * written).sum()
    version = read._version
    {"in_place": lambda: A.grad_clip([g], 1.0), "out": lambda: A.grad_clip([g], 1.0, out=[o]),
     "known": lambda: A.grad_clip([g], 1.0, total_norm=known), "list": lambda: A.grad_clip(A.grad_list([g]), 1.0),
     "allreduce": lambda: A.allreduce_clip([g, o], 1.0), "buckets": lambda: A.allreduce_clip([[o], [g]], 1.0),
     "reduce_scatter": lambda: A.allreduce_clip((g, o), 1.0, collective="reduce_scatter")}[call]()
    A.grad_norm([g, o, other])  # reads
    assert read._version == version and known._version == 0
    kept.backward()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        lost.backward()


def test_clipping_without_a_version_count():
    """Tensors made in inference mode have none."""
    A, torch = lib(), torch_mod()
    with torch.inference_mode():
        t = torch.full((3000,), 2.0, device="cuda")
        A.grad_clip([t], 1e9)
    A.grad_clip([t], math.sqrt(3000.0), eps=0.0)
    assert close(t.cpu().numpy(), np.full(3000, 1.0), 2 * U + U * U)


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P", [1, 2, 3, 4, 7, 8, 9, 17, 33])
def test_own_norms_of_long_buckets(P, dtype, kind, collective):
    """Past the sizes that are cut finer, with rank counts that fill their last batch of loads and others."""
    A, torch = lib(), torch_mod()
    sizes = [0, 200_003, 9, 70_001, 0]
    hosts = [inputs.make(dtype, P, n, seed=P + n) for n in sizes]
    op = "avg" if P % 2 else "sum"
    sums = [og.combine(x, op).astype(np.float64) for x in hosts]
    own = [og.norm_of(s, kind) for s in sums]
    norm = og.norm_of(np.array(own), kind)
    dev = [ranks_on_gpu(x, P % 3) for x in hosts]
    total, each = torch.full((), -1.0, device="cuda"), torch.full((len(sizes) + 1,), -1.0, device="cuda")
    args = (sizes, P, dtype, op, collective)
    clip = A.make_clip(kind, norm / 4, total=total, each=each)
    ws = torch.empty(A.ar_allreduce_clip_workspace_bytes(*args, clip), dtype=torch.uint8, device="cuda")
    clip.workspace, clip.workspace_bytes = ws.data_ptr(), ws.numel()
    A.ar_allreduce_clip([v for d in dev for v, _ in d], *args, clip, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert close(float(total), norm, U) and close(each[:-1].cpu().numpy(), own, U) and float(each[-1]) == -1
    f = og.factor(norm, norm / 4, 1e-6)
    for x, d, s in zip(hosts, dev, sums):
        n = x.shape[1]
        part = -(-n // P)
        for p, (view, big) in enumerate(d):
            bits = host_bits(view)
            lo, hi = (0, n) if collective == "allreduce" else (min(p * part, n), min((p + 1) * part, n))
            assert fits(bits[lo:hi], s[lo:hi] * f, dtype == "bf16"), (p, n)
            for a, b in ((0, lo), (hi, n)):
                assert np.array_equal(bits[a:b].view(np.uint8), x[p, a:b].view(np.uint8))
            assert margins_kept(big, (view.data_ptr() - big.data_ptr()) // view.element_size(), n)


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
@pytest.mark.parametrize("P,dtype", [(3, "fp32"), (2, "bf16"), (4, "bf16")])
def test_allreduce_clip_of_many_launches(P, dtype, collective):
    """More partials than the second pass joins by itself: a launch takes 16 buckets, and each has a full grid."""
    A, torch = lib(), torch_mod()
    sizes = [200_000 + i % 13 for i in range(50)]
    ranks = torch.randn(P, sum(sizes), device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    start = ranks.clone()
    buckets = [list(b) for b in zip(*(r.split(sizes) for r in ranks))]
    total = start[0].float()
    for p in range(1, P):
        total = total + start[p].float()  # rank order, fp32
    exact = total.double()
    norm = float(exact.pow(2).sum().sqrt())
    got = A.allreduce_clip(buckets, norm / 3, collective=collective)
    assert close(float(got), norm, U)
    want = exact * og.factor(norm, norm / 3, 1e-6)
    bf16 = dtype == "bf16"
    rel = (1 + 2 * U + U * U) * (1 + 2.0 ** -8) - 1 if bf16 else 2 * U + U * U
    bound = SLACK * (rel * want.abs() + (2.0 ** -134 if bf16 else 2.0 ** -150))
    rank = torch.cat([torch.arange(n, device="cuda") // -(-n // P) for n in sizes])
    for p in range(P):
        mine = (rank == p) | (collective == "allreduce")
        assert bool((((ranks[p].double() - want).abs() <= bound) | ~mine).all())
        assert bool(((ranks[p] == start[p]) | mine).all())


@pytest.mark.parametrize("collective", ["allreduce", "reduce_scatter"])
def test_kept_sums_past_32_bits(collective):
    """Sums of more than 2^32 elements that lie between the passes, with bits in both halves."""
    A, torch = lib(), torch_mod()
    n, P = (1 << 32) + 12_345, 4
    at = [0, (1 << 31) + 1, (1 << 32) + 3, n - 1]
    ranks = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(P)]
    for k, i in enumerate(at):  # 2^k (1 + 2^-8 + 2^-9): the upper half alone would round to 2^k
        for r, v in zip(ranks, (1.0, 2.0 ** -8, 2.0 ** -9, 0.0)):
            r[i] = v * 2.0 ** k
    before = [[float(r[i]) for i in at] for r in ranks]
    c = 1 + 2.0 ** -8 + 2.0 ** -9
    norm = c * math.sqrt(1 + 4 + 16 + 64)
    got = A.allreduce_clip(ranks, norm / 2, eps=0.0, collective=collective)
    assert close(float(got), norm, U)
    part = -(-n // P)
    for p, r in enumerate(ranks):
        for k, i in enumerate(at):
            mine = collective == "allreduce" or i // part == p
            # half of it, rounded up to the next bf16
            assert float(r[i]) == ((1 + 2.0 ** -7) * 2.0 ** (k - 1) if mine else before[p][k]), (p, k)
        assert int((r != 0).sum()) == sum(1 for k, i in enumerate(at) if float(r[i]) != 0)


def test_many_empty_tensors_and_buckets():
    A, torch = lib(), torch_mod()
    none = [torch.empty(0, dtype=torch.bfloat16 if i % 2 else torch.float32, device="cuda") for i in range(129)]
    for kind in ("l2", "max"):
        total, each = A.grad_norm(none, norm=kind, per_tensor=True)
        assert float(total) == 0 and each.tolist() == [0.0] * 129
        assert float(A.grad_norm(none, norm=kind)) == 0 and float(A.grad_clip(none, 1.0, norm=kind)) == 0
    assert float(A.grad_clip(none, 1.0, total_norm=torch.tensor(3.0, device="cuda"))) == 3
    for P, buckets in ((256, 2), (256, 3), (5, 20)):
        empty = [[torch.empty(0, device="cuda") for _ in range(P)] for _ in range(buckets)]
        for collective in ("allreduce", "reduce_scatter"):
            assert float(A.allreduce_clip(empty, 1.0, collective=collective)) == 0
        total, each = torch.ones((), device="cuda"), torch.ones(buckets + 1, device="cuda")
        A.ar_allreduce_clip([0] * (P * buckets), [0] * buckets, P, "fp32", "sum", "allreduce",
                            A.make_clip("l2", 1.0, total=total, each=each), torch.cuda.current_stream())
        assert float(total) == 0 and each.tolist() == [0.0] * buckets + [1.0]
