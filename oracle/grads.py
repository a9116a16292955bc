"""The global gradient norm, clipping by it, and the AdamW step.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages: after the all-reduce every replica takes its local optimizer step
on identical gradients (CS336 Lecture 8, "Data Parallelism (DDP)", step 4),
on FP32 master weights ("Distributed Training", Related, "Mixed-Precision
Training").  No page writes a clipping rule or AdamW.  Readings:

    norm = sqrt(sum of all squares)                       global 2-norm
    c    = min(1, max_norm / (norm + 1e-6))               clipping factor
    m <- b1 m + (1 - b1) g;   v <- b2 v + (1 - b2) g^2    moments
    w <- w (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)

Two forms of each: in float64, the definition; and in float32 with one
rounding per operation and the scalar factors rounded from float64 once,
which is what the HIP kernels are held to bit for bit.

Parity status: the float64 forms are pinned by the tests against PyTorch's
own clipping and AdamW run in float64, and the float32 forms against the
float64 ones within bounds derived from the count of roundings.
"""

import numpy as np


def grad_norm(tensors):
    """float64 2-norm over all elements of the tensors (float arrays)."""
    return float(np.sqrt(sum(float(np.sum(np.square(np.asarray(t, np.float64)))) for t in tensors)))


def clip_factor64(norm, max_norm):
    if np.isinf(max_norm):
        return 1.0
    c = max_norm / (norm + 1e-6)
    return 1.0 if c > 1.0 else c


def clip_factor(norm, max_norm):
    """float32, one rounding per operation; norm a float32."""
    max_norm = np.float32(max_norm)
    if np.isinf(max_norm):
        return np.float32(1)
    with np.errstate(all="ignore"):
        c = max_norm / (np.float32(norm) + np.float32(1e-6))
    return np.float32(1) if c > np.float32(1) else c


def adamw64(g, w, m, v, c, lr, b1, b2, eps, wd, t):
    """One step in float64 on float64 copies of the inputs."""
    g, w, m, v = (np.asarray(x, np.float64) for x in (g, w, m, v))
    g = c * g
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    q = m / (np.sqrt(v) / np.sqrt(1 - b2 ** t) + eps)
    return w * (1 - lr * wd) - lr / (1 - b1 ** t) * q, m, v


def adamw(g, w, m, v, c, lr, b1, b2, eps, wd, t):
    """One step in float32 as the kernel takes it: arrays float32, each
    operation rounded once; the factors float64 rounded once."""
    f = np.float32
    g, w, m, v = (np.asarray(x, f) for x in (g, w, m, v))
    s = f(lr / (1.0 - _power(b1, t)))
    r = f(1.0 / np.sqrt(1.0 - _power(b2, t)))
    with np.errstate(all="ignore"):
        g = g * f(c)
        m = f(b1) * m + f(1.0 - b1) * g
        v = f(b2) * v + f(1.0 - b2) * (g * g)
        q = m / (np.sqrt(v) * r + f(eps))
        w = w * f(1.0 - lr * wd) - s * q
    return w, m, v


def _power(b, t):
    """b^t by repeated squaring, least significant bit first, float64."""
    r = 1.0
    while t > 0:
        if t & 1:
            r *= b
        b *= b
        t >>= 1
    return r
