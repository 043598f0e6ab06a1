"""The global gradient norm, clipping and the AdamW step in 64 bits, from their formulas (numpy).
No code is shared with the GPU path. Lists of arrays of any float type, widened exactly."""

from __future__ import annotations

import numpy as np


def norm(grads, max_norm=np.inf, kind="l2", eps=1e-6, grad_scale=1.0):
    """(stats [norm, coefficient, clipped, finite], norms of the tensors)."""
    wide = [np.abs(np.asarray(g, np.float64).reshape(-1) * grad_scale) for g in grads]
    if kind == "l2":
        norms = np.array([np.sqrt(np.square(g).sum()) for g in wide])
        total = np.sqrt(np.square(norms).sum())
    else:
        norms = np.array([g.max(initial=0.0) for g in wide])
        total = norms.max()
    finite = bool(np.isfinite(total))
    coef = min(1.0, max_norm / (total + eps)) if finite else 0.0
    return np.array([total, coef, float(coef < 1.0), float(finite)]), norms


def clip(grads, max_norm, **kw):
    """(stats, norms, scaled gradients)."""
    stats, norms = norm(grads, max_norm, **kw)
    factor = stats[1] * kw.get("grad_scale", 1.0)
    return stats, norms, [np.asarray(g, np.float64) * factor if stats[3] else np.zeros(np.shape(g)) for g in grads]


def adamw(w, g, m, v, t, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, scale=1.0):
    """(weights, first moment, second moment) behind step t; scale is that of the gradient, clipping included."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    g = g * scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    # 1 - beta^t without cancellation
    c1, c2 = (-np.expm1(t * np.log(b)) if b > 0 else 1.0 for b in betas)
    return w - lr * (weight_decay * w + (m / c1) / (np.sqrt(v / c2) + eps)), m, v
