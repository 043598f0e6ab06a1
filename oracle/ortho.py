"""The orthogonalised update and the optimiser step around it, in 64 bits, from
their formulas (numpy). No code is shared with the GPU path."""

from __future__ import annotations

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(u, steps=5, coefficients=None, eps=1e-7):
    """Every singular value s of u / (|u|_F + eps) through a s + b s^3 + c s^5, `steps` times,
    by the products' definition."""
    x = np.asarray(u, np.float64)
    turned = x.shape[0] > x.shape[1]
    x = x.T if turned else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    for k in range(steps):
        a, b, c = coefficients[k] if coefficients is not None else COEFFICIENTS
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if turned else x


def newton_schulz_svd(u, steps=5, coefficients=None, eps=1e-7):
    """The same through the singular values themselves."""
    u = np.asarray(u, np.float64)
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    for k in range(steps):
        a, b, c = coefficients[k] if coefficients is not None else COEFFICIENTS
        s = a * s + b * s**3 + c * s**5
    return (left * s) @ right


def adjust_factor(rows, cols, adjust):
    return {"none": 1.0, "shape": max(1.0, rows / cols) ** 0.5, "rms": 0.2 * max(rows, cols) ** 0.5}[adjust]


def muon_step(w, g, m, lr, momentum=0.95, weight_decay=0.0, nesterov=True, adjust="shape", grad_scale=1.0, **kw):
    """(W', M') of one step."""
    g = np.asarray(g, np.float64) * grad_scale
    m = momentum * np.asarray(m, np.float64) + g
    u = g + momentum * m if nesterov else m
    w = np.asarray(w, np.float64)
    return w * (1 - lr * weight_decay) - lr * adjust_factor(*w.shape, adjust) * newton_schulz(u, **kw), m
