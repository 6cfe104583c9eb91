"""Gradient norms, clipping and the Allreduce that clips, in 64 bits (oracle).

``bits`` arguments are what the buffers hold: float32 values, or uint16 patterns of
bf16 values. Norms and factors are float64; the ranks' combination follows the
direct schedule (rank order, fp32), whose roundings are part of its definition.
"""
from __future__ import annotations

import math

import numpy as np

from .numerics import bf16_to_f32


def widen(bits: np.ndarray) -> np.ndarray:
    """fp64 values of a buffer."""
    bits = np.asarray(bits)
    return (bf16_to_f32(bits) if bits.dtype == np.uint16 else bits).astype(np.float64)


def norm_of(values: np.ndarray, kind: str) -> float:
    """Of fp64 values; NaN if any is."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    if v.size == 0:
        return 0.0
    if np.isnan(v).any():
        return math.nan
    if kind == "max":
        return float(v.max())
    top = float(v.max())
    if top == 0 or math.isinf(top):
        return top
    return top * math.sqrt(math.fsum((v / top) ** 2) if v.size <= 4096 else float(((v / top) ** 2).sum()))


def norms(tensors, kind: str):
    """(global norm, every tensor's own)."""
    each = [norm_of(widen(t), kind) for t in tensors]
    return norm_of(np.array(each), kind), np.array(each)


def factor(norm: float, max_norm: float, eps: float) -> float:
    """What a gradient of this norm is multiplied by (max_norm and eps as fp32 holds them)."""
    max_norm, eps = float(np.float32(max_norm)), float(np.float32(eps))
    reach = norm + eps
    if reach <= max_norm:
        return 1.0
    return max_norm / reach


def combine(ranks: np.ndarray, op: str) -> np.ndarray:
    """fp32 result of the ranks (first axis), added in rank order; "avg": divided once."""
    x = bf16_to_f32(ranks) if ranks.dtype == np.uint16 else np.asarray(ranks, dtype=np.float32)
    acc = x[0].copy()
    for p in range(1, x.shape[0]):
        acc = acc + x[p]
    return (acc / np.float32(x.shape[0])).astype(np.float32) if op == "avg" else acc


def allreduce_clip(buckets, max_norm: float, eps: float, op: str, kind: str):
    """(norm, factor, [fp64 scaled result of every bucket]): what every rank ends with, before rounding."""
    sums = [combine(b, op).astype(np.float64) for b in buckets]
    norm = norm_of(np.array([norm_of(s, kind) for s in sums]), kind)
    f = factor(norm, max_norm, eps)
    return norm, f, [s * f for s in sums]
