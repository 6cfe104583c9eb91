"""MI355X-native Allreduce schedules: Python side of libar_mi355x.so.

``_ar`` is the ctypes binding of include/ar.h (same function names). The
helpers below only marshal torch tensors into those calls; the product path
has no CPU fallback and fails loudly when the library is missing.
"""
from __future__ import annotations

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
def _float_types():
    import torch
    return {torch.float32: 1, torch.bfloat16: 2}  # Dtype.AR_FP32, Dtype.AR_BF16


def _invalid(message):
    return ArError(Status.AR_INVALID_ARGUMENT, message)


def _grads(tensors, out=None):
    """(GradList, device) of contiguous CUDA tensors on one device."""
    types = _float_types()
    tensors = list(tensors)
    if not tensors:
        return GradList((), 0), None
    device = tensors[0].device
    words = []
    for i, t in enumerate(tensors):
        d = types.get(t.dtype)
        if d is None or not t.is_cuda or t.device != device or not t.is_contiguous():
            raise _invalid(f"gradient {i} must be a contiguous float32 or bfloat16 tensor on {device}, a CUDA device")
        words += (t.data_ptr(), 0, t.numel(), d)
    if out is not None:
        out = list(out)
        if len(out) != len(tensors):
            raise _invalid(f"{len(tensors)} gradients, and {len(out)} outputs")
        for i, (t, o) in enumerate(zip(tensors, out)):
            d = types.get(o.dtype)
            if d is None or o.device != device or not o.is_contiguous() or o.numel() != t.numel():
                raise _invalid(f"output {i} must be a contiguous float32 or bfloat16 tensor of its gradient's size on {device}")
            words[4 * i + 1] = o.data_ptr()
            words[4 * i + 3] |= d << 32
    return GradList(words, len(tensors)), device


class _Place:
    """The device and stream of a call, with what it allocates there."""

    def __init__(self, device, stream):
        import torch
        self.torch = torch
        current = torch.cuda.current_device()
        index = current if device is None or device.index is None else device.index
        self.device = torch.device("cuda", index)
        self.guards = [] if index == current else [torch.cuda.device(index)]
        here = torch.cuda.current_stream(self.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device) if stream else torch.cuda.default_stream(self.device)
        self.stream = here if stream is None else stream
        if self.stream.device != self.device:
            raise _invalid(f"the stream is on {self.stream.device}, the gradients on {self.device}")
        if self.stream != here:  # the caller's results and the scratch belong to the stream that writes them
            self.guards.append(torch.cuda.stream(self.stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self

    def __exit__(self, *err):
        for g in reversed(self.guards):
            g.__exit__(*err)

    def floats(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.float32, device=self.device)

    def scratch(self, clip, workspace, bytes_of):
        """Point clip at the caller's workspace, or at one of torch's (in a captured call: of the graph's own memory)."""
        if workspace is None:
            workspace = self.torch.empty(bytes_of(clip), dtype=self.torch.uint8, device=self.device)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise _invalid("workspace must be a contiguous tensor on the gradients' device")
        clip.workspace, clip.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        return workspace


def grad_norm(grads, norm="l2", per_tensor=False, stream=None, workspace=None):
    """Global norm of a list of contiguous float32 / bfloat16 CUDA tensors, as a 0-dim float32 tensor.

    norm: "l2" or "max" (largest magnitude). per_tensor: return (norm, norms), norms holding
    every tensor's own. ``stream`` defaults to torch's current stream, ``workspace`` (a tensor of
    ar_grad_workspace_bytes) to scratch from torch's allocator.
    """
    table, device = _grads(grads)
    with _Place(device, stream) as at:
        total = at.floats()
        each = at.floats(table.count) if per_tensor else None
        clip = make_clip(norm, total=total, each=each)
        workspace = at.scratch(clip, workspace, lambda c: ar_grad_workspace_bytes(table, c))
        ar_grad_norm(table, clip, at.stream)
    return (total, each) if per_tensor else total


def grad_clip(grads, max_norm, norm="l2", eps=1e-6, out=None, total_norm=None, stream=None, workspace=None):
    """Scale gradients so that their global norm is at most max_norm; returns the norm before, as grad_norm does.

    scale = min(1, max_norm / (norm + eps)); in place, or into the tensors of ``out`` (same sizes,
    float32 or bfloat16). total_norm: a float32 CUDA tensor of one element that holds the norm
    already (of a gradient spread over several calls or ranks); the call then only scales.
    """
    table, device = _grads(grads, out)
    with _Place(device, stream) as at:
        if total_norm is not None:
            if total_norm.dtype != at.torch.float32 or total_norm.numel() != 1 or total_norm.device != at.device:
                raise _invalid("total_norm must be a float32 tensor of one element on the gradients' device")
            ar_grad_clip(table, make_clip(norm, max_norm, eps, known=total_norm), at.stream)
            return total_norm
        total = at.floats()
        clip = make_clip(norm, max_norm, eps, total=total)
        workspace = at.scratch(clip, workspace, lambda c: ar_grad_workspace_bytes(table, c))
        ar_grad_clip(table, clip, at.stream)
    return total


def allreduce_clip(buckets, max_norm, op="sum", norm="l2", eps=1e-6, collective="allreduce", stream=None, workspace=None):
    """In-place Allreduce of gradient buckets over P ranks, clipped by the reduced gradient's global norm.

    buckets: a list of buckets, each a list of P equally sized contiguous CUDA tensors (one per
    rank), all of one dtype (float32 or bfloat16); or one bucket's list of tensors. Ranks are combined
    in rank order, as ``allreduce(..., algo="direct")``; op "sum" or "avg". The norm (returned as a
    0-dim float32 tensor) is over all buckets, of the combined values before they are rounded;
    the scaled values are rounded once. collective "reduce_scatter": rank q ends with its part.
    """
    import torch
    buckets = list(buckets)
    if buckets and isinstance(buckets[0], torch.Tensor):
        buckets = [buckets]
    if not buckets or not len(buckets[0]):
        raise _invalid("allreduce_clip needs a bucket with a rank's tensor")
    P, first = len(buckets[0]), buckets[0][0]
    dtype = {torch.float32: Dtype.AR_FP32, torch.bfloat16: Dtype.AR_BF16}.get(first.dtype)
    if dtype is None:
        raise _invalid(f"unsupported tensor dtype {first.dtype}")
    ptrs, sizes = [], []
    for b in buckets:
        if len(b) != P:
            raise _invalid("every bucket needs a tensor of every rank")
        n = b[0].numel()
        for t in b:
            if t.dtype != first.dtype or t.numel() != n or not t.is_cuda or t.device != first.device or not t.is_contiguous():
                raise _invalid("a bucket's tensors must be contiguous CUDA tensors of one dtype, size and device")
            ptrs.append(t.data_ptr())
        sizes.append(n)
    with _Place(first.device, stream) as at:
        total = at.floats()
        clip = make_clip(norm, max_norm, eps, total=total)
        workspace = at.scratch(clip, workspace,
                               lambda c: ar_allreduce_clip_workspace_bytes(sizes, P, dtype, op, collective, c))
        ar_allreduce_clip(ptrs, sizes, P, dtype, op, collective, clip, at.stream)
    return total
