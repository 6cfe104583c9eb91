"""MI355X-native Allreduce schedules: Python side of libar_mi355x.so.

``_ar`` is the ctypes binding of include/ar.h (same function names). The
helpers below only marshal torch tensors into those calls; the product path
has no CPU fallback and fails loudly when the library is missing.
"""
from __future__ import annotations

from array import array
from operator import or_

from . import _ar
from ._ar import (  # noqa: F401
    ALGO_NAMES, ALGOS, AR_KNOB_AUTO, COLLECTIVES, COST_FORMS, DTYPES, EXECS, OPS, Algo, ArError, Collective,
    CostForm, Dtype, Exec, Kernel, Op, Schedule, Status, ar_all_gather, ar_allreduce, ar_allreduce_ex,
    ar_get_cost_model, ar_kernel_of,
    ar_last_error_message, ar_last_hip_error, ar_reduce_scatter, ar_schedule_build, ar_select, ar_set_cost_model,
    ar_set_launch_blocks, ar_status_string, ar_table_check, ar_table_check_ex, ar_version, ar_workspace_bytes,
    make_call, marshal_ptrs, ar_cache_stats_get, ar_release_cached, ar_allreduce_noalloc, AR_NOALLOC_SCRATCH_BYTES,
    AR_MAX_GRADS, GradList, NORMS, Norm, ar_allreduce_clip, ar_allreduce_clip_workspace_bytes, ar_grad_clip,
    ar_grad_norm, ar_grad_workspace_bytes, make_clip, marshal_grads,
    REDUCTIONS, Reduction, ar_vocab_loss, ar_vocab_loss_grad, ar_vocab_workspace_bytes, make_vocab,
)

_TORCH_DTYPE = {"int32": "int32", "fp32": "float32", "bf16": "bfloat16"}


def allreduce(tensors, algo="ring", op="sum", knob=0, exec="fused", batch=1, groups=None,
              stream=None, workspace=None, collective="allreduce", steps=0):
    """In-place Allreduce over a list of P equally sized CUDA tensors (one per rank).

    dtype comes from the tensors (int32, float32 or bfloat16); each tensor holds
    ``batch`` contiguous instances. ``stream`` defaults to torch's current stream.
    ``collective`` selects the reduce-scatter or all-gather half instead; ``steps``
    sets the generalized algorithm's reduction steps (0: ceil(log2 P)).
    """
    import torch

    P = len(tensors)
    t0 = tensors[0]
    rev = {v: k for k, v in _TORCH_DTYPE.items()}
    dname = str(t0.dtype).replace("torch.", "")
    if dname not in rev:
        raise ArError(Status.AR_INVALID_ARGUMENT, f"unsupported tensor dtype {t0.dtype}")
    for t in tensors:
        if t.dtype != t0.dtype or t.numel() != t0.numel() or not t.is_cuda or not t.is_contiguous():
            raise ArError(Status.AR_INVALID_ARGUMENT, "tensors must be contiguous CUDA tensors of one dtype and size")
    total = t0.numel()
    if total % batch:
        raise ArError(Status.AR_INVALID_ARGUMENT, "tensor size is not a multiple of batch")
    if stream is None:
        stream = torch.cuda.current_stream(t0.device)
    call = make_call(P, total // batch, rev[dname], op, algo, knob, exec, batch, groups,
                     workspace=workspace, workspace_bytes=(workspace.numel() * workspace.element_size()
                                                           if workspace is not None else 0),
                     collective=collective, steps=steps)
    ar_allreduce_ex(tensors, call, stream)


def reduce_scatter(tensors, algo="ring", op="sum", exec="fused", batch=1, stream=None, workspace=None):
    """In place: tensor q ends with the reduced part q (the ceil split into P parts)."""
    allreduce(tensors, algo, op, 0, exec, batch, None, stream, workspace, "reduce_scatter")


def all_gather(tensors, algo="ring", exec="fused", batch=1, stream=None, workspace=None):
    """In place: tensor q contributes part q; every tensor ends with all parts."""
    allreduce(tensors, algo, "sum", 0, exec, batch, None, stream, workspace, "all_gather")


# ---- gradient norms and clipping ----
# A call on a few small tensors takes the GPU about 5 us, so what Python does per tensor counts: the
# tensors' properties are read by maps over the unbound methods, and the common place of a call (the
# current device and stream) is found without building torch's objects for it.
_TYPES = None  # torch dtype -> ar_dtype


def _torch():
    global _TYPES
    import torch
    if _TYPES is None:
        _TYPES = {torch.float32: int(Dtype.AR_FP32), torch.bfloat16: int(Dtype.AR_BF16)}
    return torch


def _invalid(message):
    return ArError(Status.AR_INVALID_ARGUMENT, message)


def _check_tensors(torch, tensors, what):
    """(device index, ar_dtype of every tensor) of contiguous CUDA tensors on one device."""
    T = torch.Tensor
    devices = set(map(T.get_device, tensors))
    types = [_TYPES.get(t.dtype) for t in tensors]
    if len(devices) != 1 or -1 in devices or None in types or not all(map(T.is_contiguous, tensors)):
        raise _invalid(f"{what} must be contiguous float32 or bfloat16 tensors on one CUDA device")
    return devices.pop(), types


def _written(torch, tensors):
    """The kernels write through addresses: autograd, which refuses a backward pass over a saved tensor that has
    changed, learns of it here (about 50 ns a tensor)."""
    torch._C._increment_version(tensors)


def grad_list(tensors, out=None):
    """GradList of gradients, and of where a clip puts them: built once, a caller that repeats calls on tensors
    whose memory stays where it is passes it to grad_norm and grad_clip in place of the lists, which saves the
    host about 0.25 us a tensor and call. It keeps the tensors alive."""
    if isinstance(tensors, GradList):
        if out is not None:
            raise _invalid("a GradList holds its outputs already")
        return tensors
    torch = _torch()
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    count = len(tensors)
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != count:
            raise _invalid(f"{count} gradients, and {len(out)} outputs")
    if not count:
        return GradList((), 0)
    T = torch.Tensor
    index, types = _check_tensors(torch, tensors, "gradients")
    words = [0] * (4 * count)
    words[0::4] = map(T.data_ptr, tensors)
    words[2::4] = sizes = list(map(T.numel, tensors))
    if out is not None:
        there, kinds = _check_tensors(torch, out, "outputs")
        if there != index or list(map(T.numel, out)) != sizes:
            raise _invalid("every output must be of its gradient's size, on its device")
        words[1::4] = map(T.data_ptr, out)
        types = map(or_, types, map((1 << 32).__mul__, kinds))
    words[3::4] = types
    return GradList(words, count, index, (tensors, out))


class _Place:
    """The device and stream of a call, and what it allocates there."""

    def __init__(self, index, stream):
        self.torch = torch = _torch()
        current = torch.cuda.current_device()  # initializes CUDA where nothing has yet
        self.index = index = current if index is None else index
        self.guards = () if index == current else (torch.cuda.device(index),)
        self.stream = torch._C._cuda_getCurrentRawStream(index)
        if stream is None:
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
        if stream.device.index != index:
            raise _invalid(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        if stream.cuda_stream != self.stream:  # results and scratch belong to the stream that writes them
            self.guards += (torch.cuda.stream(stream),)
            self.stream = stream.cuda_stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self

    def __exit__(self, *err):
        for g in reversed(self.guards):
            g.__exit__(*err)

    def floats(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.float32, device="cuda")

    def scratch(self, clip, workspace, need, large=False):
        """Point clip at the caller's workspace. Without one, the library's own serves a call that is not captured
        (a few kB per stream, and no allocation here); otherwise need() bytes come from torch: in a captured call
        from the graph's own memory, and where they grow with the gradient (large) from memory that torch reuses."""
        if workspace is None:
            if not large and not self.torch.cuda.is_current_stream_capturing():
                return None
            size = need()
            if not size:
                return None
            workspace = self.torch.empty(size, dtype=self.torch.uint8, device="cuda")
        elif workspace.get_device() != self.index or not workspace.is_contiguous():
            raise _invalid("workspace must be a contiguous tensor on the call's device")
        clip.workspace, clip.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        return workspace


def grad_norm(grads, norm="l2", per_tensor=False, stream=None, workspace=None):
    """Global norm of a list of contiguous float32 / bfloat16 CUDA tensors (or a grad_list of them, or one tensor),
    as a 0-dim float32 tensor.

    norm: "l2" or "max" (largest magnitude). per_tensor: return (norm, norms), norms holding
    every tensor's own. Norms carry no gradient. ``stream`` defaults to torch's current stream (results
    are ready on the stream that is given), ``workspace`` (a tensor of ar_grad_workspace_bytes) to the
    library's own or, in a captured call, to memory of the graph.
    """
    table = grad_list(grads)
    with _Place(table.index, stream) as at:
        total = at.floats()
        each = at.floats(table.count) if per_tensor else None
        clip = make_clip(norm, total=total, each=each)
        workspace = at.scratch(clip, workspace, lambda: ar_grad_workspace_bytes(table, clip))
        ar_grad_norm(table, clip, at.stream)
    return (total, each) if per_tensor else total


def grad_clip(grads, max_norm, norm="l2", eps=1e-6, out=None, total_norm=None, stream=None, workspace=None):
    """Scale gradients so that their global norm is at most max_norm; returns the norm before, as grad_norm does.

    scale = min(1, max_norm / (norm + eps)); in place, or into the tensors of ``out`` (same sizes,
    float32 or bfloat16). total_norm: a float32 CUDA tensor of one element that holds the norm
    already (of a gradient spread over several calls or ranks), apart from what the call writes; the call then
    only scales.
    """
    table = grad_list(grads, out)
    with _Place(table.index, stream) as at:
        if total_norm is not None:
            if total_norm.dtype != at.torch.float32 or total_norm.numel() != 1 or total_norm.get_device() != at.index:
                raise _invalid("total_norm must be a float32 tensor of one element on the gradients' device")
            total = total_norm
            ar_grad_clip(table, make_clip(norm, max_norm, eps, known=total), at.stream)
        else:
            total = at.floats()
            clip = make_clip(norm, max_norm, eps, total=total)
            workspace = at.scratch(clip, workspace, lambda: ar_grad_workspace_bytes(table, clip))
            ar_grad_clip(table, clip, at.stream)
        if table.tensors:
            grads, out = table.tensors
            _written(at.torch, grads if out is None else out)
    return total


def allreduce_clip(buckets, max_norm, op="sum", norm="l2", eps=1e-6, collective="allreduce", stream=None, workspace=None):
    """In-place Allreduce of gradient buckets over P ranks, clipped by the reduced gradient's global norm.

    buckets: a list of buckets, each a list of P equally sized contiguous CUDA tensors (one per
    rank), all of one dtype (float32 or bfloat16); or one bucket's list of tensors. Ranks are combined
    in rank order, as ``allreduce(..., algo="direct")``; op "sum" or "avg". The norm (returned as a
    0-dim float32 tensor) is over all buckets, of the combined values before they are rounded;
    scale and product are fp32 values, and a bf16 result is rounded from the product. collective
    "reduce_scatter": rank q ends with its part.
    """
    torch = _torch()
    T = torch.Tensor
    buckets = list(buckets)
    if buckets and isinstance(buckets[0], T):
        buckets = [buckets]
    P = len(buckets[0]) if buckets else 0
    if not P or any(len(b) != P for b in buckets):
        raise _invalid("allreduce_clip needs buckets with a tensor of every rank")
    tensors = buckets[0] if len(buckets) == 1 else [t for b in buckets for t in b]
    index, types = _check_tensors(torch, tensors, "the ranks' tensors")
    numels = list(map(T.numel, tensors))
    sizes = numels[::P]
    if numels != (sizes * P if len(sizes) == 1 else [n for n in sizes for _ in range(P)]) or len(set(types)) != 1:
        raise _invalid("a bucket's tensors must be of one size, and all tensors of one dtype")
    args = sizes, P, types[0], _ar._enum(OPS, op), _ar._enum(COLLECTIVES, collective)
    with _Place(index, stream) as at:
        total = at.floats()
        clip = make_clip(norm, max_norm, eps, total=total)
        workspace = at.scratch(clip, workspace, lambda: ar_allreduce_clip_workspace_bytes(*args, clip),
                               large=args[4] == Collective.AR_REDUCE_SCATTER)
        ar_allreduce_clip(array("Q", map(T.data_ptr, tensors)), *args, clip, at.stream)
        _written(torch, tensors)
    return total


# ---- losses over a vocabulary in pieces ----
def _rows(torch, t, what, dtype, index):
    """(address, distance of rows) of a matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype != dtype or t.get_device() != index:
        raise _invalid(f"{what} must be a matrix of {dtype} on cuda:{index}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise _invalid(f"{what}'s rows must be contiguous")
    return t.data_ptr(), t.stride(0)


def _outputs(torch, given, like, what, index):
    if given is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if not isinstance(given, torch.Tensor) or given.shape != like.shape:
        raise _invalid(f"{what} must be of its gradient's shape")
    return given


def _vocab(hidden, weight, ids, logits, reduction, ignore_index, temperature, token_weights, grad, out_hidden,
           out_weight, stream, workspace):
    torch = _torch()
    single = isinstance(weight, torch.Tensor)
    pieces = [weight] if single else list(weight)
    if not isinstance(hidden, torch.Tensor) or hidden.dtype not in _TYPES or not hidden.is_cuda or hidden.dim() != 2:
        raise _invalid("hidden must be a float32 or bfloat16 matrix on a CUDA device")
    T, H = hidden.shape
    index, dtype = hidden.get_device(), hidden.dtype
    place, ld = _rows(torch, hidden, "hidden", dtype, index)
    table = []
    for w in pieces:
        at, wld = _rows(torch, w, "every piece of the output matrix", dtype, index)
        if w.shape[1] != H:
            raise _invalid("hidden and the output matrix differ in width")
        table.append([at, None, w.shape[0], wld, 0])
    shape = (T,) if logits is None else (T, logits.shape[1] if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 0)
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64) or ids.get_device() != index \
            or tuple(ids.shape) != shape or (T and shape[-1] > 1 and ids.stride(-1) != 1):
        raise _invalid("targets must be int32 or int64, one a token (a teacher's ids: as many as its logits, in "
                       "contiguous rows), on hidden's device")
    kw = {}
    if logits is not None:
        if not shape[1] or logits.dtype not in _TYPES:
            raise _invalid("teacher logits must be a float32 or bfloat16 matrix of at least one column")
        at, lld = _rows(torch, logits, "teacher logits", logits.dtype, index)
        kw = dict(top=shape[1], logits=at, logits_ld=lld, logits_dtype=_TYPES[logits.dtype], ids_ld=ids.stride(0))
    w = token_weights
    if w is not None and (not isinstance(w, torch.Tensor) or w.dtype != torch.float32 or w.get_device() != index
                          or tuple(w.shape) != (T,) or not w.is_contiguous()):
        raise _invalid("token_weights must be contiguous float32, one a token, on hidden's device")
    if reduction not in REDUCTIONS:
        raise _invalid(f"reduction must be one of {', '.join(REDUCTIONS)}")
    with _Place(index, stream) as at:
        each = reduction == "none"
        loss = at.floats(T) if each else at.floats()
        d_hidden = d_weights = None
        if grad:
            d_hidden = _outputs(torch, out_hidden, hidden, "out_hidden", index)
            kw["dh"], kw["dh_ld"] = _rows(torch, d_hidden, "out_hidden", dtype, index)
            outs = [None] * len(pieces) if out_weight is None else [out_weight] if single else list(out_weight)
            if len(outs) != len(pieces):
                raise _invalid(f"{len(pieces)} pieces, and {len(outs)} outputs")
            d_weights = [_outputs(torch, o, w, "out_weight", index) for o, w in zip(outs, pieces)]
            for row, d in zip(table, d_weights):
                row[1], row[4] = _rows(torch, d, "out_weight", dtype, index)
        call = make_vocab(T, H, _TYPES[dtype], place, ld, [tuple(row) for row in table], ids.data_ptr(),
                          loss.data_ptr(), temperature=temperature, reduction=reduction, ids_bytes=ids.element_size(),
                          ignore=ignore_index,
                          token_weights=None if token_weights is None else token_weights.data_ptr(), **kw)
        workspace = at.scratch(call, workspace, lambda: ar_vocab_workspace_bytes(call, grad), large=True)
        (ar_vocab_loss_grad if grad else ar_vocab_loss)(call, at.stream)
        if grad:
            _written(torch, [d_hidden] + d_weights)
    return (loss, d_hidden, d_weights[0] if single else d_weights) if grad else loss


def vocab_loss(hidden, weight, targets, reduction="mean", ignore_index=-100, temperature=1.0, token_weights=None,
               stream=None, workspace=None):
    """Softmax cross entropy of hidden states against a vocabulary in pieces, without keeping the logits.

    hidden: [T, H], float32 or bfloat16; weight: the output matrix [V, H] of the same type, or the list of its
    pieces [V_p, H] in rank order (rows contiguous, any distance apart); targets: [T], int32 or int64. Logits are
    hidden weight^T / temperature. Rows whose target is ignore_index are left out (loss 0); an id outside the
    vocabulary makes the loss NaN. token_weights: float32 [T], each row's factor. reduction: "mean" (over the rows
    that are not left out, whatever their weight; 0 if there are none) and "sum" give a 0-dim float32 tensor,
    "none" every row's loss. Losses carry no autograd history: vocab_loss_grad gives the gradients.
    ``stream`` defaults to torch's current stream, ``workspace`` (ar_vocab_workspace_bytes) to memory from torch.
    """
    return _vocab(hidden, weight, targets, None, reduction, ignore_index, temperature, token_weights, False, None, None,
                  stream, workspace)


def vocab_loss_grad(hidden, weight, targets, reduction="mean", ignore_index=-100, temperature=1.0, token_weights=None,
                    out_hidden=None, out_weight=None, stream=None, workspace=None):
    """vocab_loss and its gradients: (loss, d_hidden, d_weight), d_weight as weight (a tensor, or a list of pieces).

    The gradients are of the loss ("none": of the rows' sum), in the inputs' type; d_hidden is the sum over all
    pieces, as an Allreduce of the ranks' parts leaves it. out_hidden, out_weight: tensors that receive them. The
    workspace holds up to 4 GiB of logits at a time (2 bytes each in bf16, 10 in fp32).
    """
    return _vocab(hidden, weight, targets, None, reduction, ignore_index, temperature, token_weights, True, out_hidden,
                  out_weight, stream, workspace)


def distill_loss(hidden, weight, teacher_logits, teacher_ids, reduction="mean", temperature=1.0, token_weights=None,
                 stream=None, workspace=None):
    """Distance of a student to a teacher's top logits, over a vocabulary in pieces, without the student's logits.

    teacher_logits: [T, K], float32 or bfloat16, and teacher_ids: [T, K], int32 or int64; a negative id ends or
    thins out a row's list, and a row without entries is left out. With q the softmax of a row's teacher logits /
    temperature and p that of hidden weight^T / temperature over the whole vocabulary, the row's loss is
    sum_k q_k (log q_k - log p_id(k)) (no factor of temperature squared). The other arguments as for vocab_loss.
    """
    return _vocab(hidden, weight, teacher_ids, _given(teacher_logits), reduction, 0, temperature, token_weights, False,
                  None, None, stream, workspace)


def distill_loss_grad(hidden, weight, teacher_logits, teacher_ids, reduction="mean", temperature=1.0,
                      token_weights=None, out_hidden=None, out_weight=None, stream=None, workspace=None):
    """distill_loss and its gradients, as vocab_loss_grad gives them. The teacher's logits get none."""
    return _vocab(hidden, weight, teacher_ids, _given(teacher_logits), reduction, 0, temperature, token_weights, True,
                  out_hidden, out_weight, stream, workspace)


def _given(logits):
    if logits is None:
        raise _invalid("teacher logits are missing")
    return logits
