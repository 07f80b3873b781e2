"""CPU oracle of the Muon step on Shard(0) shards (test infrastructure only).

Plain NumPy, sharing no code with the HIP library.  The elementwise steps
compute in fp32, one IEEE round-to-nearest operation at a time in the order of
the C header; the orthogonalisation in fp64 from its definition.
"""
from __future__ import annotations

from typing import List, Sequence

import numpy as np

from .fsdp import Plan, bf16_rne, bf16_to_f32, reduce

F32 = np.float32


def _segment(p: Plan, shards: Sequence[np.ndarray]) -> np.ndarray:
    out = np.zeros(p.S, dtype=np.uint16)
    for e, x in zip(p.entries, shards):
        out[e.shard_offset:e.shard_offset + e.valid_numel] = bf16_rne(x)
    return out


def momentum(p: Plan, grads: Sequence[np.ndarray], ms: Sequence[np.ndarray], mu: float,
             nesterov: bool) -> np.ndarray:
    """m = mu*m + (1-mu)*g in place; returns the bf16 segment of the updates."""
    a, b = F32(mu), F32(1.0 - mu)
    us: List[np.ndarray] = []
    with np.errstate(all="ignore"):
        for g, m in zip(grads, ms):
            h = b * g
            m[...] = a * m + h
            us.append(a * m + h if nesterov else m.copy())
    return _segment(p, us)


def reduce_momentum(p: Plan, rs_in: np.ndarray, ms: Sequence[np.ndarray], mu: float,
                    nesterov: bool) -> np.ndarray:
    return momentum(p, reduce(p, rs_in), ms, mu, nesterov)


def update(p: Plan, masters: Sequence[np.ndarray], upd: Sequence[np.ndarray],
           scales: Sequence[float], lr: float, weight_decay: float) -> np.ndarray:
    """p = p*(1-lr*wd) - (lr*s)*o in place; returns the bf16 copy-in segment.
    upd: each parameter's bf16 bits of o for this rank's valid elements."""
    decay = F32(1.0 - lr * weight_decay)
    with np.errstate(all="ignore"):
        for x, o, s in zip(masters, upd, scales):
            step = F32(lr) * F32(s)
            x[...] = x * decay - step * bf16_to_f32(o)
    return _segment(p, masters)


def orthogonalize(u: np.ndarray, coeffs: Sequence[Sequence[float]], eps: float = 1e-7) -> np.ndarray:
    """The Newton-Schulz iterate in fp64: X0 = U / (|U|_F + eps), then for each
    (a, b, c): X <- a X + b (X X^T) X + c (X X^T)^2 X on the smaller side."""
    x = u.astype(np.float64)
    if x.size == 0:
        return x
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    with np.errstate(all="ignore"):
        x = x / (np.sqrt((x * x).sum()) + eps)
        for a, b, c in coeffs:
            g = x @ x.T
            x = a * x + (b * g + c * (g @ g)) @ x
    return np.ascontiguousarray(x.T if tall else x)
