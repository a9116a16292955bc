"""The gradient norm, clipping, all-reduce with norm and AdamW step on the
GPU: the norm against float64 within one rounding, everything else bit for
bit against the oracle's float32 forms (themselves held to float64 on the
CPU)."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_helpers import DEV, assert_same_bits, oracle_ring, to_device, to_host, torch_dtype

pytestmark = pytest.mark.gpu
ddp = pytest.importorskip("gradient_all_reduce_allreduce_amd")

TILE = 16384                      # bytes of one norm or clip tile
# (The norm's, for sets past 64 pieces of 4 KiB: of these "many" and "long".  The
# clip's is 4 KiB, AdamW's 256 elements.  test_gpu_grads_paths.py has the ends of
# the tiles on every path.)
SIZES = {
    "one": [1],
    "few": [5, 1, 0, 33, 4097],
    "tiles": [TILE // 4 - 1, TILE // 4, TILE // 4 + 1, TILE // 2, 3 * TILE // 2 + 3],
    "many": [1 + 37 * k % 1500 for k in range(800)],      # several launches
    "long": [2_500_003, 7],
}


def draw(numels, dtype, scale=0.01, seed=0):
    """Host arrays (float32 values; bf16 ones representable) and each one's
    type; "mixed" alternates."""
    rng = np.random.default_rng(seed)
    out, types = [], []
    for t, n in enumerate(numels):
        x = (rng.standard_normal(n) * scale * 2.0 ** rng.integers(-4, 5)).astype(np.float32)
        kind = ("bf16", "f32")[t % 2] if dtype == "mixed" else dtype
        if kind == "bf16":
            x = oracle.bf16_bits_to_f32(oracle.f32_to_bf16_bits(x))
        out.append(x)
        types.append(kind)
    return out, types


class Arena:
    """Tensors at chosen element offsets of one guarded buffer each type:
    gap elements of a canary between them, which nothing may change."""
    CANARY = 0x5A

    def __init__(self, arrays, types, gap=3):
        self.held, self.views, self.used = {}, [], {}
        for kind in set(types):
            total = sum(len(a) + gap for a, k in zip(arrays, types) if k == kind) + gap
            es = 2 if kind == "bf16" else 4
            self.held[kind] = torch.full((total * es,), self.CANARY, dtype=torch.uint8, device=DEV).view(torch_dtype(kind))
            self.used[kind] = gap
        self.at = []
        for a, kind in zip(arrays, types):
            o = self.used[kind]
            v = self.held[kind][o:o + len(a)]
            v.copy_(torch.from_numpy(a))
            self.views.append(v)
            self.at.append((kind, o, len(a)))
            self.used[kind] += len(a) + gap

    def host(self):
        return [v.float().cpu().numpy() for v in self.views]

    def check_canaries(self):
        for kind, x in self.held.items():
            es = 2 if kind == "bf16" else 4
            b = x.view(torch.uint8).cpu().numpy().copy().reshape(-1, es)
            for k, o, n in self.at:
                if k == kind:
                    b[o:o + n] = self.CANARY
            assert (b == self.CANARY).all(), f"bytes outside the {kind} tensors changed"


def separate(arrays, types):
    return [torch.from_numpy(a).to(DEV).to(torch_dtype(k)) for a, k in zip(arrays, types)]


def check_norm(got, arrays):
    want = oracle.grad_norm(arrays)
    n = sum(a.size for a in arrays)
    # one rounding to float32; float64 sums lose at most n steps
    assert abs(float(got) - want) <= (2.0 ** -24 + n * 2.0 ** -53) * want, (float(got), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES)
def test_norm(sizes, dtype):
    arrays, types = draw(SIZES[sizes], dtype)
    sep = ddp.MultiGrad(separate(arrays, types))
    a = sep.norm()
    check_norm(a, arrays)
    assert a.shape == () and a.dtype == torch.float32
    assert torch.equal(a, sep.norm()), "same tensors, same bits"
    arena = Arena(arrays, types)
    check_norm(ddp.grad_norm(arena.views), arrays)
    arena.check_canaries()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_extreme_values(dtype):
    big = 2.0 ** 127
    for value, n in ((big, 3), (2.0 ** -126, 1000), (2.0 ** -133, 70_000), (0.0, 100)):
        x = torch.full((n,), value, dtype=torch_dtype(dtype), device=DEV)
        got = float(ddp.grad_norm(x))
        want = float(np.float32(np.sqrt(float(n)) * value))
        assert got == pytest.approx(want, rel=2.0 ** -23, abs=0)
    assert float(ddp.grad_norm(torch.full((9,), big, device=DEV))) == float("inf")     # 3 * 2^127
    x = torch.ones(5000, dtype=torch_dtype(dtype), device=DEV)
    for k in (0, 4999):
        for bad in (float("inf"), float("-inf")):
            y = x.clone()
            y[k] = bad
            assert float(ddp.grad_norm([x, y])) == float("inf")
        y = x.clone()
        y[k] = float("nan")
        assert np.isnan(float(ddp.grad_norm([x, y])))
        y[k - 1] = float("inf")
        assert np.isnan(float(ddp.grad_norm([x, y])))


def test_norm_counts_a_tensor_as_often_as_it_is_listed():
    x = torch.full((16,), 3.0, device=DEV)
    assert float(ddp.grad_norm([x, x, x, x])) == 24.0


def test_norm_of_empty_tensors_is_zero():
    empty = torch.zeros(0, device=DEV)
    assert float(ddp.grad_norm([empty, empty])) == 0.0
    assert float(ddp.clip_grads([empty], 1.0)) == 0.0


def test_long_tensor_past_32_bits():
    """2^31 + 1001 bf16 elements (byte offsets past 2^32): values at the
    ends and around the 2^31st element only."""
    n = 2 ** 31 + 1001
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    marks = [0, 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31, n - 1]
    for k, i in enumerate(marks):
        x[i] = float(2 ** k)
    want = np.sqrt(sum(4.0 ** k for k in range(len(marks))))
    norm = ddp.clip_grads(x, float(np.float32(want)) / 2)
    assert abs(float(norm) - want) <= 2.0 ** -24 * want * (1 + 1e-6)
    c = oracle.clip_factor(np.float32(float(norm)), float(np.float32(want)) / 2)
    assert int(torch.count_nonzero(x)) == len(marks)
    for k, i in enumerate(marks):
        assert float(x[i]) == float(oracle.bf16_bits_to_f32(
            oracle.f32_to_bf16_bits(np.asarray([c * np.float32(2 ** k)], np.float32)))[0])


# ------------------------------------------------------------------ clip ----

def clipped(arrays, types, norm, max_norm):
    c = oracle.clip_factor(norm, max_norm)
    out = []
    with np.errstate(all="ignore"):
        for a, k in zip(arrays, types):
            y = a * c
            out.append(oracle.bf16_bits_to_f32(oracle.f32_to_bf16_bits(y)) if k == "bf16" else y)
    return out


def same(got, want, what=""):
    assert len(got) == len(want)
    for t, (g, w) in enumerate(zip(got, want)):
        assert_same_bits(g.astype(np.float32), w.astype(np.float32), f"{what} tensor {t}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES)
def test_clip(sizes, dtype):
    arrays, types = draw(SIZES[sizes], dtype)
    half = 0.5 * oracle.grad_norm(arrays)
    # into other tensors that lie at other offsets
    src, dst = Arena(arrays, types, gap=3), Arena([np.zeros_like(a) for a in arrays], types, gap=5)
    norm = ddp.clip_grads(src.views, half, out=dst.views)
    check_norm(norm, arrays)
    assert torch.equal(norm, ddp.grad_norm(src.views)), "the norm's own call gives the same bits"
    want = clipped(arrays, types, np.float32(float(norm)), half)
    same(dst.host(), want, "out")
    same(src.host(), arrays, "inputs")
    # in place, separate tensors; the same norm, bit for bit
    sep = separate(arrays, types)
    check_norm(ddp.clip_grads(sep, half), arrays)
    # in place, in the arena, the norm given
    given = torch.tensor(7.25, device=DEV)
    assert ddp.clip_grads(src.views, 2.0, norm=given) is given and float(given) == 7.25
    same(src.host(), clipped(arrays, types, np.float32(7.25), 2.0), "given")
    src.check_canaries()
    dst.check_canaries()


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_below_the_limit_keeps_every_bit(dtype, inplace):
    arrays, types = draw(SIZES["tiles"], dtype)
    ts = separate(arrays, types)
    out = None if inplace else [torch.full_like(t, 9.0) for t in ts]
    for limit in (1e9, float("inf")):
        ddp.clip_grads(ts, limit, out=out)
        same([t.float().cpu().numpy() for t in out or ts], arrays)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_of_subnormal_values(dtype):
    """Values over the whole exponent range: products that underflow are
    rounded into the subnormals, not flushed."""
    rng = np.random.default_rng(3)
    a = (rng.standard_normal(9001) * np.exp2(rng.integers(-149, -90, 9001))).astype(np.float32)
    if dtype == "bf16":
        a = oracle.bf16_bits_to_f32(oracle.f32_to_bf16_bits(a))
    for n in (9001, 400_000):            # one workgroup, and many
        arrays, types = [np.resize(a, n)], [dtype]
        ts = separate(arrays, types)
        ddp.clip_grads(ts, 1.0, norm=torch.tensor(3.7, device=DEV))
        same([t.float().cpu().numpy() for t in ts], clipped(arrays, types, np.float32(3.7), 1.0))
        ts = separate(arrays, types)
        norm = ddp.clip_grads(ts, 1e-30)
        check_norm(norm, arrays)
        same([t.float().cpu().numpy() for t in ts], clipped(arrays, types, np.float32(float(norm)), 1e-30))


def test_clip_special_norms():
    """What the documentation says of norms that are not finite, and of a
    limit of zero."""
    x = torch.tensor([1.0, -2.0, float("inf"), 4.0], device=DEV)
    norm = ddp.clip_grads(x, 1.0)
    assert float(norm) == float("inf")
    got = x.cpu().numpy()
    assert (got[[0, 1, 3]] == 0).all() and np.isnan(got[2])
    x = torch.tensor([1.0, float("nan")], device=DEV)
    assert np.isnan(float(ddp.clip_grads(x, 1.0))) and torch.isnan(x).all()
    x = torch.tensor([3.0, -4.0], device=DEV)
    ddp.clip_grads(x, 0.0)
    assert (x == 0).all()
    x = torch.tensor([3.0, float("inf")], device=DEV)
    ddp.clip_grads(x, float("inf"))
    assert x.cpu().tolist() == [3.0, float("inf")]
    x = torch.zeros(3, device=DEV)
    ddp.clip_grads(x, 1.0)
    assert (x == 0).all()


def test_clip_refuses_the_same_tensor_twice_in_place():
    x = torch.ones(64, device=DEV)
    with pytest.raises(ddp.DdpError):
        ddp.clip_grads([x, x], 1.0)
    with pytest.raises(ddp.DdpError):
        ddp.clip_grads([x, x[10:20]], 1.0)
    with pytest.raises(ValueError):
        ddp.clip_grads([x], 1.0, out=[torch.ones(64, dtype=torch.bfloat16, device=DEV)])
    with pytest.raises(ValueError):
        ddp.clip_grads([x], 1.0, out=[torch.ones(63, device=DEV)])
    with pytest.raises(ValueError):
        ddp.clip_grads([torch.ones(8, 8, device=DEV).t()], 1.0)
    with pytest.raises(TypeError):
        ddp.grad_norm(torch.ones(4, dtype=torch.float16, device=DEV))
    assert (x == 1).all()


# ----------------------------------------------------------------- adamw ----

H = dict(lr=3e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
ADAMW_SIZES = {
    "few": [5, 1, 0, 33, 4097],
    "tiles": [2047, 2048, 2049, 4096, 6145],
    "many": [1 + 37 * k % 700 for k in range(400)],       # several launches
    "long": [1_500_003, 7],
}


def state(arrays, seed, zero=False):
    w, _ = draw([a.size for a in arrays], "f32", 0.02, seed)
    m, _ = draw([a.size for a in arrays], "f32", 1e-3, seed + 1)
    v, _ = draw([a.size for a in arrays], "f32", 1e-2, seed + 2)
    return w, [x * (not zero) for x in m], [x * x * (not zero) for x in v]


def adamw_want(arrays, w, m, v, c, t, h=H):
    steps = [oracle.adamw(*x, c, h["lr"], h["b1"], h["b2"], h["eps"], h["wd"], t) for x in zip(arrays, w, m, v)]
    return [[s[k] for s in steps] for k in range(3)]


def adamw_run(call, t, norm=None, max_norm=None, h=H):
    call(h["lr"], t, betas=(h["b1"], h["b2"]), eps=h["eps"], weight_decay=h["wd"], norm=norm, max_norm=max_norm)


def as_bf16(x):
    return oracle.bf16_bits_to_f32(oracle.f32_to_bf16_bits(x))


@pytest.mark.parametrize("params", [None, "f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", ADAMW_SIZES)
def test_adamw(sizes, dtype, params):
    arrays, types = draw(ADAMW_SIZES[sizes], dtype)
    w, m, v = state(arrays, 10)
    f32 = ["f32"] * len(arrays)
    # every stream at offsets of its own
    G, W, M, V = Arena(arrays, types, 3), Arena(w, f32, 1), Arena(m, f32, 2), Arena(v, f32, 5)
    P = Arena([np.zeros_like(a) for a in arrays], [params] * len(arrays), 7) if params else None
    norm = torch.tensor(3.5, device=DEV)
    adamw_run(ddp.MultiGrad(G.views).bind_adamw(W.views, M.views, V.views, P.views if P else None), 7, norm, 1.25)
    ww, wm, wv = adamw_want(arrays, w, m, v, oracle.clip_factor(np.float32(3.5), 1.25), 7)
    same(W.host(), ww, "w")
    same(M.host(), wm, "m")
    same(V.host(), wv, "v")
    same(G.host(), arrays, "gradients")
    if P:
        same(P.host(), [as_bf16(x) for x in ww] if params == "bf16" else ww, "params")
    for a in (G, W, M, V) + ((P,) if P else ()):
        a.check_canaries()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adamw_steps_from_zero_moments_like_torchs(dtype):
    """Ten steps without a norm; the step count once as an int and once on
    the GPU give the same bits, and torch's own AdamW in float64 the same
    weights within the float32 roundings: 10 steps of at most 2^-24 * |w| *
    3 each and updates of at most lr (1 + wd) whose terms are off by under
    2^-16 of that bound (m off by up to 36 roundings of the largest g over
    ten steps, g / sqrt(v) up to 4.5, some 50 more in the quotient)."""
    arrays0, types = draw([3001, 17], dtype)
    w, m, v = state(arrays0, 20, zero=True)
    a = [separate(x, ["f32"] * 2) for x in (w, m, v)]
    b = [separate(x, ["f32"] * 2) for x in (w, m, v)]
    p = [torch.nn.Parameter(torch.from_numpy(x.astype(np.float64))) for x in w]
    opt = torch.optim.AdamW(p, lr=H["lr"], betas=(H["b1"], H["b2"]), eps=H["eps"], weight_decay=H["wd"])
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    for t in range(1, 11):
        arrays, _ = draw([3001, 17], dtype, seed=30 + t)
        g = separate(arrays, types)
        count += 1
        adamw_run(ddp.MultiGrad(g).bind_adamw(*a), t)
        adamw_run(ddp.MultiGrad(g).bind_adamw(*b), count)
        w, m, v = adamw_want(arrays, w, m, v, np.float32(1), t)
        for x, y in zip(p, arrays):
            x.grad = torch.from_numpy(y.astype(np.float64))
        opt.step()
    for k, want in enumerate((w, m, v)):
        same([x.cpu().numpy() for x in a[k]], want)
        same([x.cpu().numpy() for x in b[k]], want)
    for x, y in zip(p, w):
        np.testing.assert_allclose(y, x.detach().numpy(), rtol=30 * 2.0 ** -24, atol=10 * H["lr"] * 1.1 * 2.0 ** -16)


def test_adamw_leaves_a_step_out():
    """A norm that is not finite, or a count on the GPU below 1: nothing
    changes, the copy of the weights included."""
    arrays, types = draw([5000, 3], "f32")
    w, m, v = state(arrays, 40)
    g = separate(arrays, types)
    st = [separate(x, types) for x in (w, m, v)]
    par = [torch.full_like(x, 7.0) for x in st[0]]
    run = ddp.MultiGrad(g).bind_adamw(*st, params=par)
    for bad in (float("inf"), float("nan")):
        adamw_run(run, 3, torch.tensor(bad, device=DEV), 1.0)
    adamw_run(run, torch.zeros(1, dtype=torch.int64, device=DEV))
    for k, want in enumerate((w, m, v)):
        same([x.cpu().numpy() for x in st[k]], want)
    assert all((x == 7).all() for x in par)
    # a limit without bound never scales
    adamw_run(run, 3, torch.tensor(50.0, device=DEV), float("inf"))
    same([x.cpu().numpy() for x in st[0]], adamw_want(arrays, w, m, v, np.float32(1), 3)[0])


def test_adamw_special_values():
    """Infinite and NaN gradients without a norm follow IEEE; zero gradients
    with zero moments and eps = 0 give 0 / 0."""
    g = np.array([np.inf, -np.inf, np.nan, 0.0, 1e30, 1e-30], np.float32)
    w, m, v = (np.full(6, x, np.float32) for x in (0.5, 0.0, 0.0))
    for eps in (1e-8, 0.0):
        st = [torch.from_numpy(x.copy()).to(DEV) for x in (w, m, v)]
        h = dict(H, eps=eps)
        adamw_run(ddp.MultiGrad(torch.from_numpy(g).to(DEV)).bind_adamw(*st), 1, h=h)
        want = adamw_want([g], [w], [m], [v], np.float32(1), 1, h)
        same([x.cpu().numpy() for x in st], [x[0] for x in want])


def test_adamw_over_the_whole_exponent_range():
    """Gradients and state from subnormal to huge: subnormals are kept, the
    division and root are rounded correctly everywhere."""
    rng = np.random.default_rng(9)
    n = 50_000

    def wide(lo, hi):
        return (rng.standard_normal(n) * np.exp2(rng.integers(lo, hi, n))).astype(np.float32)
    g, w, m = wide(-149, 60), wide(-149, 100), wide(-149, 100)
    v = np.abs(wide(-149, 100))
    for eps in (1e-8, 0.0, 1e-40):
        st = [torch.from_numpy(x.copy()).to(DEV) for x in (w, m, v)]
        h = dict(H, eps=eps)
        adamw_run(ddp.MultiGrad(torch.from_numpy(g).to(DEV)).bind_adamw(*st), 3, torch.tensor(2.5, device=DEV), 1.0, h)
        want = adamw_want([g], [w], [m], [v], oracle.clip_factor(np.float32(2.5), 1.0), 3, h)
        same([x.cpu().numpy() for x in st], [x[0] for x in want], f"eps {eps}")


def test_adamw_refusals():
    x = [torch.zeros(8, device=DEV) for _ in range(4)]
    mg = ddp.MultiGrad(x[0])
    with pytest.raises(ValueError):
        mg.bind_adamw(x[1], x[2], torch.zeros(9, device=DEV))
    with pytest.raises(TypeError):
        mg.bind_adamw(x[1], x[2], torch.zeros(8, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        mg.bind_adamw([x[1], x[1]], x[2], x[3])
    run = mg.bind_adamw(*x[1:])
    with pytest.raises(ValueError):
        run(1e-3, 1, norm=torch.tensor(1.0, device=DEV))
    with pytest.raises(ValueError):
        run(1e-3, 1, max_norm=1.0)
    with pytest.raises(ValueError):
        run(1e-3, torch.ones(1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        run(1e-3, 1, norm=torch.tensor(1.0), max_norm=1.0)
    with pytest.raises(ddp.DdpError):
        run(1e-3, 0)
    with pytest.raises(ddp.DdpError):
        mg.bind_adamw(x[1], x[1], x[3])(1e-3, 1)
    with pytest.raises(ValueError):
        ddp.MultiGrad([x[0], x[1].bfloat16()]).bind_adamw(x[:2], x[:2], x[:2])


def test_adamw_past_32_bit_offsets():
    """2^30 + 77 elements: float32 offsets pass 2^32 bytes.  Sampled blocks
    against the oracle."""
    n = 2 ** 30 + 77
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    w, m, v = (torch.zeros(n, device=DEV) for _ in range(3))
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    places = [0, 2 ** 29 - 50, 2 ** 30 - 50, n - 100]
    for k, o in enumerate(places):
        arrays, _ = draw([100], "bf16", seed=50 + k)
        s = state(arrays, 60 + k)
        for x, y in zip((g, w, m, v), (arrays, *s)):
            x[o:o + 100] = torch.from_numpy(y[0]).to(DEV)
    # (the last two blocks share elements: what lies there once all are set)
    parts = [[[x[o:o + 100].float().cpu().numpy()] for x in (g, w, m, v)] for o in places]
    adamw_run(ddp.MultiGrad(g).bind_adamw(w, m, v, p), 5)
    for o, part in zip(places, parts):
        want = adamw_want(*part, np.float32(1), 5)
        for x, y in zip((w, m, v), want):
            same([x[o:o + 100].cpu().numpy()], y)
        same([p[o:o + 100].float().cpu().numpy()], [as_bf16(want[0][0])])
    assert int(torch.count_nonzero(m)) <= 400


# --------------------------------------------------------- all-reduce norm ----

def rank_draw(P, n, dtype, seed):
    X = workloads.rank_buffers(P, n, "wide", 1.0, seed=seed)
    return workloads.to_bf16_bits(X) if dtype == "bf16" else X


@pytest.mark.parametrize("pair", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("P,n,C,op", [(1, 1000, 1, "sum"), (2, 70_001, 2, "mean"), (3, 5, 3, "mean"),
                                      (8, 300_007, 8, "mean"), (8, 1, 8, "sum"), (8, 4096, 64, "sum"),
                                      (16, 20_003, 16, "mean"), (5, 100_000, 10, "sum")])
def test_allreduce_norm(P, n, C, op, pair):
    it, ot = pair
    X = rank_draw(P, n, it, seed=n)
    ins = to_device(X, it)
    want = oracle_ring(X, op, C, in_dtype=it, out_dtype=ot)
    out, norm = ddp.allreduce_norm(ins, op, C, out_dtype=torch_dtype(ot))
    assert_same_bits(to_host(out), want, "outputs")
    one = torch.full((n + 8,), 9.0, dtype=torch_dtype(ot), device=DEV)
    got, norm1 = ddp.allreduce_norm(ins, op, C, out=[one[:n]])
    assert len(got) == 1
    assert_same_bits(to_host([one[:n]]), want[:1], "one copy")
    assert (one[n:] == 9).all()
    assert_same_bits(to_host(ins), X, "inputs")
    row = oracle.bf16_bits_to_f32(want[0]) if ot == "bf16" else want[0]
    check_norm(norm, [row])
    check_norm(norm1, [row])


@pytest.mark.parametrize("P,C,E,n", [(8, 8, 8192, 3 * 8192 + 1000), (8, 8, 32768, 3 * 32768 + 12347),
                                     (4, 4, 1000, 5 * 1000 + 3), (2, 3, 512, 2000), (8, 8, 65536, 65536)])
@pytest.mark.parametrize("copies", ["ranks", "one"])
def test_allreduce_norm_buckets(P, C, E, n, copies):
    X = rank_draw(P, n, "f32", seed=n)
    want = np.concatenate([oracle_ring(X[:, lo:lo + E], "mean", C) for lo in range(0, n, E)], axis=1)
    ins = to_device(X, "f32")
    out = ins if copies == "ranks" else [ins[0]]            # in place
    got, norm = ddp.allreduce_norm(ins, "mean", C, out=out, bucket_elems=E)
    assert_same_bits(to_host(got), want[:len(out)], "buckets")
    check_norm(norm, [want[0]])


def test_allreduce_norm_many_partials():
    """Past 4,096 workgroups the sum has a second level."""
    P, n = 8, 256 * 17_000 + 100
    X = rank_draw(P, n, "bf16", seed=3)
    out, norm = ddp.allreduce_norm(to_device(X, "bf16"), "mean", P, out_dtype=torch.float32)
    want = oracle_ring(X, "mean", P, in_dtype="bf16", out_dtype="f32")
    assert_same_bits(to_host(out), want)
    check_norm(norm, [want[0]])


def test_allreduce_norm_over_several_launches():
    """2^29 + 777 elements go out as two launches whose partial sums lie
    behind each other; the outputs are the plain call's."""
    P, n = 2, 2 ** 29 + 777
    rows = []
    for r in range(P):
        x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
        x[::4097] = float(r + 1)
        x[-5:] = 3.0
        rows.append(x)
    one = torch.empty(n, device=DEV)
    _, norm = ddp.allreduce_norm(rows, "sum", P, out=[one])
    want = torch.empty(n, device=DEV)
    ddp.allreduce(rows, "sum", P, out=[want, torch.empty(n, device=DEV)])
    assert torch.equal(one, want)
    exact = float(one.double().square().sum().sqrt())
    assert abs(float(norm) - exact) <= 2.0 ** -24 * exact * (1 + 1e-6)


def test_allreduce_norm_replayed():
    """A captured call (two launches, the second counting its workgroups from
    a word the first clears) replayed with new gradients, eager calls of the
    same sizes between."""
    P, n = 4, 256 * 5000 + 3
    rows = [torch.empty(n, device=DEV) for _ in range(P)]
    one = torch.empty(n, device=DEV)
    for r in rows:
        r.normal_()
    ddp.allreduce_norm(rows, "mean", P, out=[one])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, norm = ddp.allreduce_norm(rows, "mean", P, out=[one])
    for t in range(1, 5):
        for r in rows:
            r.normal_().mul_(t)
        graph.replay()
        got = one.clone(), norm.clone()
        out, eager = ddp.allreduce_norm(rows, "mean", P)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out[0]) and torch.equal(got[0], out[P - 1])
        assert torch.equal(got[1], eager)
        check_norm(eager, [out[0].cpu().numpy()])


def test_allreduce_norm_nothing_and_not_finite():
    empty = [torch.zeros(0, device=DEV) for _ in range(2)]
    out, norm = ddp.allreduce_norm(empty)
    assert float(norm) == 0.0
    rows = [torch.ones(1000, device=DEV) for _ in range(2)]
    rows[1][999] = float("inf")
    assert float(ddp.allreduce_norm(rows)[1]) == float("inf")
    rows[0][999] = float("-inf")
    assert np.isnan(float(ddp.allreduce_norm(rows)[1]))


# ------------------------------------------------- streams, graphs, chains ----

def test_on_another_stream_and_two_at_once():
    """One MultiGrad on two streams at the same time: each call has a
    workspace of its own."""
    arrays, types = draw([3_000_001, 5, 400_000], "f32")
    mg = ddp.MultiGrad(separate(arrays, types))
    out = [torch.empty_like(g) for g in mg.grads]
    want = mg.norm()
    s = [torch.cuda.Stream() for _ in range(2)]
    run = mg.bind_clip(out)
    torch.cuda.synchronize()
    got = []
    for k in range(20):
        with torch.cuda.stream(s[k % 2]):
            got.append(mg.norm() if k % 2 else run(0.5))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    same([o.cpu().numpy() for o in out], clipped(arrays, types, np.float32(float(want)), 0.5))


def test_with_another_gpu_current(monkeypatch):
    """A call that finds another GPU current makes the tensors' one current
    for its launches (seen from one GPU: the first question is answered
    wrongly, the results are the same)."""
    arrays, types = draw([300_000, 5], "f32")
    g = separate(arrays, types)
    w, m, v = state(arrays, 90)
    st = [separate(x, types) for x in (w, m, v)]
    mg = ddp.MultiGrad(g)
    out = [torch.empty_like(x) for x in g]
    clip, step = mg.bind_clip(out), mg.bind_adamw(*st)
    rows = [torch.ones(1000, device=DEV) for _ in range(2)]
    real, wrong, asked = torch.cuda.current_device, [], []

    def current():
        asked.append(bool(wrong))
        return wrong.pop() if wrong else real()
    monkeypatch.setattr(torch.cuda, "current_device", current)
    norms = []
    for call in (mg.norm, lambda: clip(0.5), lambda: adamw_run(step, 2), lambda: ddp.allreduce_norm(rows)[1]):
        wrong.append(real() + 1)
        norms.append(call())
        assert not wrong and asked[-1] is False
    monkeypatch.undo()
    check_norm(norms[0], arrays)
    assert torch.equal(norms[0], norms[1]) and float(norms[3]) == np.float32(np.sqrt(4000.0))
    same([x.cpu().numpy() for x in out], clipped(arrays, types, np.float32(float(norms[1])), 0.5))
    same([x.cpu().numpy() for x in st[0]], adamw_want(arrays, w, m, v, np.float32(1), 2)[0])


def test_allreduce_norm_same_bits_at_every_cap():
    """The cap on resident workgroups is a launch shape: outputs and norm keep
    their bits."""
    X = rank_draw(8, 300_007, "bf16", seed=11)
    first = None
    try:
        for cap in (-1, 0, 2, 7, 16):
            ddp.ddp_set_wg_per_cu("ring", cap)
            out, norm = ddp.allreduce_norm(to_device(X, "bf16"), "mean", 8, out_dtype=torch.float32)
            first = first or (out[3], norm)
            assert torch.equal(out[3], first[0]) and torch.equal(norm, first[1])
    finally:
        ddp.ddp_set_wg_per_cu("ring", -1)


def test_graphs_replayed_between_eager_calls():
    """Two graphs of the same MultiGrad, each a clip and a step whose count
    lives on the GPU, replayed in turn with eager calls between."""
    arrays, types = draw([50_001, 300, 7], "f32", 0.1)
    g = separate(arrays, types)
    w, m, v = state(arrays, 70, zero=True)
    st = [separate(x, types) for x in (w, m, v)]
    mg = ddp.MultiGrad(g)
    out = [torch.empty_like(x) for x in g]
    clip, step = mg.bind_clip(out), ddp.MultiGrad(out).bind_adamw(*st)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # warm-up outside the graphs
        clip(1.0)
    torch.cuda.current_stream().wait_stream(side)
    graphs, norms = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            count.add_(1)
            norms.append(clip(1.0))
            adamw_run(step, count)
        graphs.append(graph)
    for t in range(1, 7):
        new, _ = draw([50_001, 300, 7], "f32", 0.1, seed=80 + t)
        for x, y in zip(g, new):
            x.copy_(torch.from_numpy(y))
        graphs[t % 2].replay()
        eager = mg.norm()
        torch.cuda.synchronize()
        assert torch.equal(norms[t % 2], eager)
        cl = clipped(new, types, np.float32(float(eager)), 1.0)
        same([x.cpu().numpy() for x in out], cl, f"replay {t}")
        w, m, v = adamw_want(cl, w, m, v, np.float32(1), t)
        for x, y in zip(st, (w, m, v)):
            same([z.cpu().numpy() for z in x], y, f"replay {t}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_steps_all_reduce_norm_clip_adamw(dtype):
    """Three data-parallel steps as they are used: bucketed all-reduce of the
    ranks' gradients with its norm into one copy, AdamW clipped by it on
    views of the flat buffers, against the oracle chain; and the same through
    clipping every rank's copy first."""
    P, E = 4, 8192
    shapes = [(70, 100), (33,), (1,), (128, 129), (5, 7, 11)]
    plan = ddp.GradBucketer(shapes, torch_dtype(dtype), E * (2 if dtype == "bf16" else 4))
    n = plan.total
    arena = plan.alloc_arena(P)
    rows = [arena[r, :n] for r in range(P)]
    w, m, v = plan.alloc_state(3)
    w0 = workloads.rank_buffers(1, n, "normal", 0.02, seed=5)[0]
    hw, hm, hv = w0, np.zeros(n, np.float32), np.zeros(n, np.float32)
    w.copy_(torch.from_numpy(w0))
    m.zero_()
    v.zero_()
    grad = torch.empty(n, device=DEV)
    params = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    views = [plan.tensor_views(x) for x in (grad, w, m, v, params)]
    mg = ddp.MultiGrad(views[0])
    step = mg.bind_adamw(*views[1:4], params=views[4])
    for t in range(1, 4):
        X = workloads.rank_buffers(P, n, "normal", 0.05, seed=t)
        X = workloads.to_bf16_bits(X) if dtype == "bf16" else X
        for r, x in enumerate(to_device(X, dtype)):
            rows[r].copy_(x)
        _, norm = ddp.allreduce_norm(rows, "mean", P, out=[grad], bucket_elems=E)
        adamw_run(step, t, norm, 1.0)
        want = np.concatenate([oracle_ring(X[:, lo:lo + E], "mean", P, in_dtype=dtype, out_dtype="f32")[0]
                               for lo in range(0, n, E)])
        assert_same_bits(to_host([grad])[0], want, "reduced")
        check_norm(norm, [want])
        c = oracle.clip_factor(np.float32(float(norm)), 1.0)
        assert c < 1
        hw, hm, hv = oracle.adamw(want, hw, hm, hv, c, H["lr"], H["b1"], H["b2"], H["eps"], H["wd"], t)
        for x, y in ((w, hw), (m, hm), (v, hv)):
            assert_same_bits(x.cpu().numpy(), y, f"step {t}")
        assert_same_bits(params.float().cpu().numpy(), as_bf16(hw), "params")
        # every rank's copy, clipped in place by the norm the all-reduce left
        out, norm2 = ddp.allreduce_norm(rows, "mean", P, out=rows, bucket_elems=E)
        before = to_host(rows)
        ddp.clip_grads(rows, 1.0, norm=norm2)
        wide = [oracle.bf16_bits_to_f32(b) if dtype == "bf16" else b for b in before]
        got = [r.float().cpu().numpy() for r in rows]
        same(got, clipped(wide, [dtype] * P, np.float32(float(norm2)), 1.0), "rows")
