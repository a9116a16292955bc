"""Pins of the oracle's norm, clipping and AdamW: the float64 forms against
torch's own in float64, the float32 forms against the float64 ones."""

import numpy as np
import pytest
import torch

import oracle

U = 2.0 ** -24        # half a step of float32, relative


def draw(n, scale, seed):
    return (np.random.default_rng(seed).standard_normal(n) * scale).astype(np.float32)


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 3.0, 1e6])
def test_clip_is_torchs(max_norm):
    ts = [draw(n, 0.3, n) for n in (1, 7, 100, 1000)]
    ps = [torch.nn.Parameter(torch.zeros(t.size, dtype=torch.float64)) for t in ts]
    for p, t in zip(ps, ts):
        p.grad = torch.from_numpy(t.astype(np.float64))
    norm = torch.nn.utils.clip_grad_norm_(ps, max_norm)
    assert abs(float(norm) - oracle.grad_norm(ts)) <= 1e-14 * oracle.grad_norm(ts)
    c = oracle.clip_factor64(oracle.grad_norm(ts), max_norm)
    for p, t in zip(ps, ts):
        np.testing.assert_allclose(p.grad.numpy(), c * t.astype(np.float64), rtol=1e-14, atol=0)


def test_clip_factor_of_special_norms():
    inf = float("inf")
    assert oracle.clip_factor(inf, 1.0) == 0 and np.isnan(oracle.clip_factor(float("nan"), 1.0))
    assert oracle.clip_factor(0.0, 1.0) == 1 and oracle.clip_factor(0.0, 0.0) == 0
    assert oracle.clip_factor(inf, inf) == 1 and oracle.clip_factor(2.0, inf) == 1
    for norm in (0.3, 1.0, 7.7, 1e9):
        want = oracle.clip_factor64(float(np.float32(norm)), 0.9)
        assert abs(float(oracle.clip_factor(norm, 0.9)) - want) <= 5 * U * want


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_adamw64_is_torchs(wd):
    w0, n = draw(257, 0.02, 1), 257
    p = torch.nn.Parameter(torch.from_numpy(w0.astype(np.float64)))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=wd)
    w, m, v = w0.astype(np.float64), np.zeros(n), np.zeros(n)
    for t in range(1, 6):
        g = draw(n, 0.01, 100 + t)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        w, m, v = oracle.adamw64(g, w, m, v, 1.0, 3e-3, 0.9, 0.95, 1e-8, wd, t)
        np.testing.assert_allclose(p.detach().numpy(), w, rtol=1e-12, atol=1e-15)


def adamw_bounds(g, w, m, v, c, lr, b1, b2, eps, wd, t):
    """How far the float32 step may be from the float64 one, from the count
    of roundings (U each, all terms of v positive): c itself 2 and its product
    1; m: b1 m 2 and the sum 1, (1 - b1) g 2 + 3 and the sum 1; v: 2 * 3 + 1
    for g^2, 2 for the factor, 1 for the sum; the denominator half of v's 10,
    then 1 for the root, 2 for r and its product, 1 for eps' sum; the
    quotient 1, lr's factor and its product 2; the decayed w 2, the result 1."""
    w1, m1, v1 = oracle.adamw64(g, w, m, v, c, lr, b1, b2, eps, wd, t)
    g, w, m = (np.abs(np.asarray(x, np.float64)) for x in (g, w, m))
    dm = U * (3 * b1 * m + 6 * (1 - b1) * c * g)
    den = np.sqrt(v1) / np.sqrt(1 - b2 ** t) + eps
    s = lr / (1 - b1 ** t)
    dw = U * (2 * w * (1 - lr * wd) + np.abs(w1)) + s * (dm / den + U * 12 * np.abs(m1) / den)
    tiny = 2.0 ** -126            # products that underflow lose up to a subnormal's step
    return 1.01 * dw + tiny, 1.01 * dm + tiny, 1.01 * 10 * U * v1 + tiny


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 6])
@pytest.mark.parametrize("max_norm", [1e6, 0.3])
def test_adamw32_is_within_its_roundings(t, max_norm):
    n = 20_000
    g, w = draw(n, 0.01, 2), draw(n, 0.02, 3)
    m = draw(n, 1e-3, 4) if t > 1 else np.zeros(n, np.float32)
    v = draw(n, 1e-2, 5) ** 2 if t > 1 else np.zeros(n, np.float32)
    norm = np.float32(oracle.grad_norm([g]))
    h = (3e-4, 0.9, 0.999, 1e-8, 0.1, t)
    got = oracle.adamw(g, w, m, v, oracle.clip_factor(norm, max_norm), *h)
    c = oracle.clip_factor64(float(norm), max_norm)
    want = oracle.adamw64(g, w, m, v, c, *h)
    for a, b, d in zip(got, want, adamw_bounds(g, w, m, v, c, *h)):
        assert a.dtype == np.float32
        assert np.all(np.abs(a.astype(np.float64) - b) <= d)
