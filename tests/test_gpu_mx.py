"""4-bit gradients, their all-reduce and AdamW with 8-bit moments on the GPU,
bit for bit against the oracle; norms within one rounding of float64, the
weights of AdamW within the roundings that the oracle counts."""

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import DEV, assert_same_bits, torch_dtype
from oracle import mx

pytestmark = pytest.mark.gpu
ddp = pytest.importorskip("gradient_all_reduce_allreduce_amd")

f = np.float32
NS = [1, 7, 8, 31, 32, 33, 511, 512, 513, 1000, 4099, 70_001]


def rounded(x, kind):
    x = np.asarray(x, f)
    return oracle.bf16_bits_to_f32(oracle.f32_to_bf16_bits(x)) if kind == "bf16" else x


def values(n, kind, seed=0, scale=1e-2):
    """Values whose blocks differ by many powers of two, zeros and whole zero
    blocks among them, and many on the levels' borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(n) * scale * 2.0 ** rng.integers(-20, 20, -(-n // 32)).repeat(32)[:n]
    x[rng.random(n) < 0.05] = 0
    x[(np.arange(n) // 32) % 11 == 5] = 0
    border = rng.random(n) < 0.2
    x[border] = (rng.integers(-28, 29, n) * 0.25 * 2.0 ** rng.integers(-12, -8, n))[border]
    return rounded(x, kind)


class Guarded:
    """Values of a type at an element offset of a buffer of their own, with a
    canary before and behind them that nothing may change."""
    BYTE = 0x5A

    def __init__(self, array, kind, offset=0):
        dtype = {"u8": torch.uint8}.get(kind) or torch_dtype(kind)
        x = torch.from_numpy(np.ascontiguousarray(array)).to(dtype)
        self.n, self.offset, self.es = x.numel(), offset + 64, x.element_size()
        self.held = torch.full(((self.n + self.offset + 64) * self.es,), self.BYTE, dtype=torch.uint8, device=DEV)
        self.view = self.held.view(dtype)[self.offset:self.offset + self.n]
        self.view.copy_(x)

    def host(self):
        return self.view.cpu().numpy() if self.es == 1 else self.view.float().cpu().numpy()

    def intact(self):
        b = self.held.cpu().numpy()
        lo = self.offset * self.es
        assert (b[:lo] == self.BYTE).all() and (b[lo + self.n * self.es:] == self.BYTE).all(), "bytes outside changed"


def guarded_mx(n, offset=0):
    blocks = -(-n // 32)
    codes, scales = Guarded(np.full(blocks * 16, 0x33), "u8"), Guarded(np.full(blocks, 0x44), "u8", offset)
    return codes, scales, ddp.Mx4(codes.view, scales.view, n)


def bits(x):
    return np.ascontiguousarray(x).view(np.uint32)


# ------------------------------------------------------------ quantise ----

def check_quantize(P, n, kind, left_kind, offset=0, arrays=None, lefts=None):
    arrays = arrays if arrays is not None else [values(n, kind, seed=r) for r in range(P)]
    if lefts is None and left_kind:
        lefts = [values(n, left_kind, seed=100 + r, scale=1e-3) for r in range(P)]
    g = [Guarded(a, kind, offset) for a in arrays]
    left = [Guarded(a, left_kind, offset) for a in lefts] if left_kind else None
    out = [guarded_mx(n, offset) for _ in range(P)]
    got = ddp.mx4_quantize([x.view for x in g], residual=[x.view for x in left] if left else None,
                           out=[x[2] for x in out])
    torch.cuda.synchronize()
    for r in range(P):
        codes, scales, new = mx.mx4_quantize(arrays[r], lefts[r] if left_kind else None)
        assert np.array_equal(out[r][1].host(), scales), (r, "scales")
        assert np.array_equal(out[r][0].host(), codes), (r, "codes")
        assert_same_bits(g[r].host(), arrays[r], "gradients unchanged")
        if left_kind:
            assert_same_bits(left[r].host(), rounded(new, left_kind), f"residual of rank {r}")
            left[r].intact()
        for x in (g[r], out[r][0], out[r][1]):
            x.intact()
    return got


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("left_kind", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize(kind, left_kind, n):
    check_quantize(3, n, kind, left_kind)


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 8, 13])
@pytest.mark.parametrize("kind,left_kind", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_quantize_anywhere(kind, left_kind, offset):
    check_quantize(2, 1537, kind, left_kind, offset)


@pytest.mark.parametrize("left_kind", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("P, n", [(1, 2 ** 20), (1, 2 ** 20 + 1), (2, 2 ** 19 + 513), (3, 350_213)])
def test_quantize_long(P, n, kind, left_kind):
    """Up to 2^20 elements in all a wave takes one span, over that two."""
    check_quantize(P, n, kind, left_kind, offset=1)


@pytest.mark.parametrize("P", [1, 2, 5, 16])
def test_quantize_ranks(P):
    check_quantize(P, 2050, "f32", "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_every_border(kind):
    """Every level, every border between two and the float32 next to both, in
    every exponent that a scale can have, both signs."""
    points = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5], f)
    points = np.concatenate([points, np.nextafter(points, f(9)), np.nextafter(points, f(-9))])
    rows = []
    for k in range(-126, 126):
        for part in points.reshape(-1, 16):
            rows.append(np.concatenate([part, -part[:15], [6]]) * 2.0 ** k)
    x = rounded(np.concatenate(rows), kind)
    check_quantize(1, x.size, kind, None, arrays=[x])
    check_quantize(1, x.size, kind, "f32", arrays=[x], lefts=[np.zeros_like(x)])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_over_the_exponent_range(kind):
    """A block's maximum at and next to every power of two and 1.75 of it, down
    to the subnormals, up to what has no scale; infinities and NaN."""
    tops = [m * 2.0 ** k for k in range(-149, 128) for m in (1, 1.5, 1.75, 1.875) if m * 2.0 ** k < 3.4e38]
    tops = np.array(tops, f)
    with np.errstate(over="ignore"):
        tops = np.concatenate([tops, np.nextafter(tops, f(np.inf)), np.nextafter(tops, f(0)),
                               np.array([np.inf, -np.inf, np.nan, 3.4e38, -3.4e38], f)])
    x = np.zeros((tops.size, 32), f)
    with np.errstate(all="ignore"):
        for e in range(32):
            x[:, e] = tops * f([1, 0.9, 0.3, -0.1, 0.02, -1, 0.25, 0.5][e % 8])
    x = x[:, np.random.default_rng(0).permutation(32)]
    x = rounded(x.reshape(-1), kind)
    lefts = np.where(np.arange(x.size) % 7 == 0, 0, np.minimum(np.abs(np.nan_to_num(x, posinf=1, neginf=1)), 1e30) / 16)
    check_quantize(1, x.size, kind, "f32", arrays=[x], lefts=[lefts.astype(f)])
    check_quantize(1, x.size, kind, None, arrays=[x])


def test_quantize_a_bucket_of_its_own():
    n, E = 5000, 1024
    plan = ddp.GradBucketer([(n,)], torch.float32, E * 4)
    x = torch.from_numpy(values(n, "f32")).to(DEV)
    whole = plan.alloc_mx4(1)
    parts = plan.alloc_mx4(1)
    ddp.mx4_quantize([x], out=whole)
    for b in range(plan.n_buckets):
        lo = b * E
        ddp.mx4_quantize([x[lo:lo + plan.bucket_len(b)]], out=[parts[0].narrow(lo, plan.bucket_len(b))])
    assert torch.equal(whole[0].codes, parts[0].codes) and torch.equal(whole[0].scales, parts[0].scales)


def test_quantize_nothing():
    x = torch.zeros(0, device=DEV)
    got = ddp.mx4_quantize([x, x], residual=[x, x])
    assert got[0].numel == 0 and ddp.mx4_dequantize(got)[1].numel() == 0
    out, norm = ddp.allreduce_mx4_norm(got, "mean")
    assert out[0].numel() == 0 and float(norm) == 0.0


def test_rows_past_32_bit_offsets():
    """2^32 + 1001 elements: blocks at both ends and around each 2^31st
    element against the oracle, through quantisation, the all-reduce of the
    row with itself and reading back."""
    n = 2 ** 32 + 1001
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    places = [0, 2 ** 31 - 4096, 2 ** 32 - 4096]         # the last one to the end
    want = {}
    for k, at in enumerate(places):
        count = min(8192, n - at)
        a = values(count, "bf16", seed=k)
        x[at:at + count] = torch.from_numpy(a).to(DEV)
        want[at] = a
    coded = ddp.mx4_quantize([x])
    del x
    twice = ddp.allreduce_mx4([coded[0], coded[0]], "sum", out=[torch.empty(n, dtype=torch.bfloat16, device=DEV)])[0]
    for at, a in want.items():
        codes, scales, _ = mx.mx4_quantize(a)
        q = mx.mx4_decode(codes, scales, a.size)
        assert_same_bits(twice[at:at + a.size].float().cpu().numpy(), 2 * q, f"at {at}")
    del twice
    back = ddp.mx4_dequantize(coded, dtype=torch.bfloat16)[0]
    for at, a in want.items():
        codes, scales, _ = mx.mx4_quantize(a)
        assert_same_bits(back[at:at + a.size].float().cpu().numpy(), mx.mx4_decode(codes, scales, a.size), f"at {at}")
        assert not back[at + 8192:at + 8192 + 100].any()


# ---------------------------------------------------------- dequantise ----

def any_codes(n, seed=0, special=True):
    """Every code under every scale byte, 0 and 255 among them."""
    rng = np.random.default_rng(seed)
    blocks = -(-n // 32)
    scales = rng.integers(0 if special else 60, 256 if special else 190, blocks).astype(np.uint8)
    return rng.integers(0, 256, blocks * 16).astype(np.uint8), scales


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 3])
def test_dequantize(kind, n, offset):
    P = 2
    coded = [any_codes(n, seed=r) for r in range(P)]
    rows = [ddp.Mx4(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), n) for c, s in coded]
    out = [Guarded(np.zeros(n, f), kind, offset) for _ in range(P)]
    ddp.mx4_dequantize(rows, out=[o.view for o in out])
    torch.cuda.synchronize()
    for r, (c, s) in enumerate(coded):
        assert_same_bits(out[r].host(), rounded(mx.mx4_decode(c, s, n), kind), f"row {r}")
        out[r].intact()


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), 256 // 16 * 16)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16)
    n = scales.size * 32
    codes = codes[:n // 2]
    row = ddp.Mx4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), n)
    assert_same_bits(ddp.mx4_dequantize([row])[0].cpu().numpy(), mx.mx4_decode(codes, scales, n))


# ---------------------------------------------------------- all-reduce ----

def on_gpu(coded, n):
    return [ddp.Mx4(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), n) for c, s in coded]


def check_norm(got, written):
    x = np.asarray(written, np.float64)
    want = np.sqrt(np.square(x).sum())
    assert abs(float(got) - want) <= (2.0 ** -24 + x.size * 2.0 ** -53) * want


def check_reduce(P, n, op, kind, copies, seed=0, offset=0):
    coded = [any_codes(n, seed=seed + r, special=False) for r in range(P)]
    want = rounded(mx.mx4_allreduce(np.stack([mx.mx4_decode(c, s, n) for c, s in coded]), op), kind)
    rows = on_gpu(coded, n)
    out = [Guarded(np.zeros(n, f), kind, offset) for _ in range(copies)]
    got, norm = ddp.allreduce_mx4_norm(rows, op, out=[o.view for o in out])
    for o in out:
        assert_same_bits(o.host(), want, f"P={P} n={n}")
        o.intact()
    check_norm(norm, want)
    plain = ddp.allreduce_mx4(rows, op, out=[torch.empty(n, dtype=torch_dtype(kind), device=DEV) for _ in range(copies)])
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


@pytest.mark.parametrize("P", range(1, 17))
@pytest.mark.parametrize("op", ["sum", "mean"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_allreduce(P, op, kind):
    check_reduce(P, 1300, op, kind, P)
    check_reduce(P, 77, op, kind, 1)


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_allreduce_lengths(n, kind):
    check_reduce(4, n, "sum", kind, 4, offset=n % 7)
    check_reduce(3, n, "mean", kind, 1, offset=1)


@pytest.mark.parametrize("P", [3, 5, 6, 7, 9, 10, 11, 12, 13, 14, 15])
@pytest.mark.parametrize("low, high", [(0, 6), (10, 30), (100, 104), (90, 130), (248, 255)])
def test_mean_is_the_nearest_float32(P, low, high):
    """Where quotients are subnormal, ordinary and where sums are infinite."""
    n = 1 << 15
    rng = np.random.default_rng(P)
    coded = [(rng.integers(0, 256, n // 2).astype(np.uint8), rng.integers(low, high, n // 32).astype(np.uint8))
             for _ in range(P)]
    with np.errstate(all="ignore"):
        want = mx.mx4_allreduce(np.stack([mx.mx4_decode(c, s, n) for c, s in coded]), "mean")
    assert_same_bits(ddp.allreduce_mx4(on_gpu(coded, n), "mean")[0].cpu().numpy(), want)


LONG = 2 ** 22        # elements from which a wave takes more than one span


@pytest.mark.parametrize("P", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("tail", [1, 513, 2049 + 512, 8191])
def test_long_rows_are_their_parts(P, tail):
    """A row long enough for waves of several spans, and its parts, which are
    not: the same codes, values and left-overs, and nothing behind the row."""
    n = LONG + tail
    rng = np.random.default_rng(P)
    coded = [(rng.integers(0, 256, -(-n // 32) * 16).astype(np.uint8),
              rng.integers(90, 130, -(-n // 32)).astype(np.uint8)) for _ in range(P)]
    rows = on_gpu(coded, n)
    parts = [(0, LONG // 2), (LONG // 2, n - LONG // 2)]
    for copies in {1, P}:
        out = [guarded_mx(n, 1) for _ in range(copies)]
        coded_out, norm = ddp.allreduce_mx4_norm(rows, "mean", out=[x[2] for x in out])
        values16 = [Guarded(np.zeros(n, f), "bf16", 1) for _ in range(copies)]
        _, norm16 = ddp.allreduce_mx4_norm(rows, "mean", out=[x.view for x in values16])
        check_norm(norm, ddp.mx4_dequantize(coded_out[:1])[0].cpu().numpy())
        check_norm(norm16, values16[0].host())
        for at, length in parts:
            mine = [r.narrow(at, length) for r in rows]
            want = ddp.allreduce_mx4(mine, "mean", out=[ddp.Mx4.empty(length)])[0]
            want16 = ddp.allreduce_mx4(mine, "mean", out=[torch.empty(length, dtype=torch.bfloat16, device=DEV)])[0]
            for k in range(copies):
                got = out[k][2].narrow(at, length)
                assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales), (copies, at)
                assert torch.equal(values16[k].view[at:at + length], want16), (copies, at)
        for x in out:
            x[0].intact(), x[1].intact()
        for x in values16:
            x.intact()


def test_allreduce_norm_of_many_workgroups():
    check_reduce(2, 5_000_011, "mean", "f32", 1)


def check_coded(P, n, op, copies, left_kind, in_place=False, seed=0):
    coded = [any_codes(n, seed=seed + r, special=False) for r in range(P)]
    g = mx.mx4_allreduce(np.stack([mx.mx4_decode(c, s, n) for c, s in coded]), op)
    left0 = values(n, left_kind, seed=9) if left_kind else None
    codes, scales, new = mx.mx4_quantize(g, left0)
    rows = on_gpu(coded, n)
    left = Guarded(left0, left_kind, 3) if left_kind else None
    guards = [guarded_mx(n, 1) for _ in range(copies)]
    out = rows[:copies] if in_place else [x[2] for x in guards]
    got, norm = ddp.allreduce_mx4_norm(rows, op, out=out, residual=left.view if left else None)
    for o in got:
        assert np.array_equal(o.codes.cpu().numpy(), codes) and np.array_equal(o.scales.cpu().numpy(), scales)
    for x in guards:
        x[0].intact(), x[1].intact()
    if left_kind:
        assert_same_bits(left.host(), rounded(new, left_kind), "residual")
        left.intact()
    check_norm(norm, mx.mx4_decode(codes, scales, n))


@pytest.mark.parametrize("left_kind", [None, "f32", "bf16"])
@pytest.mark.parametrize("P", [1, 2, 3, 8, 13, 16])
def test_allreduce_coded(P, left_kind):
    for n in (1, 33, 512, 1543):
        check_coded(P, n, "mean", P, left_kind)
        check_coded(P, n, "sum", 1, left_kind)


@pytest.mark.parametrize("copies", [1, 4])
def test_allreduce_coded_in_place(copies):
    check_coded(4, 3001, "mean", copies, "f32", in_place=True)


def test_allreduce_of_blocks_without_numbers():
    n = 200
    coded = [any_codes(n, seed=r, special=False) for r in range(3)]
    coded[1][1][2] = 255
    rows = on_gpu(coded, n)
    out, norm = ddp.allreduce_mx4_norm(rows, "mean")
    assert torch.isnan(norm)
    for o in out:
        nan = torch.isnan(o).cpu().numpy()
        assert nan[64:96].all() and nan.sum() == 32
    left = torch.full((n,), 0.5, device=DEV)
    again = ddp.allreduce_mx4(rows, "mean", out=[ddp.Mx4.empty(n, DEV)], residual=left)[0]
    assert again.scales[2] == 255 and not again.codes[32:48].any() and (left[64:96] == 0.5).all()
    assert (again.scales[[0, 1, 3, 4, 5, 6]] != 255).all()


def test_allreduce_rounds_in_rank_order():
    """1 + 2^-24 - 1 in float32 is 0 in rank order and 2^-24 in another."""
    rows = []
    for level, s in ((2, 127), (2, 103), (10, 127)):       # code 2 is 1, code 10 is -1
        rows.append((np.full(16, level | level << 4, np.uint8), np.array([s], np.uint8)))
    out = ddp.allreduce_mx4(on_gpu(rows, 32), "sum")[0]
    assert not out.any()
    out = ddp.allreduce_mx4(on_gpu([rows[0], rows[2], rows[1]], 32), "sum")[0]
    assert (out == 2.0 ** -24).all()


# --------------------------------------------------------------- AdamW ----

HYPER = dict(lr=1e-2, b1=0.9, b2=0.99, eps=1e-8, wd=0.1)
SIZES = {"one": [1], "few": [5, 1, 0, 33, 4097], "tiles": [255, 256, 257, 511, 512, 513, 1025],
         "many": [1 + 37 * k % 700 for k in range(300)], "long": [600_011, 7]}


def moments(n, seed):
    rng = np.random.default_rng(seed)
    return mx.moments_encode(values(n, "f32", seed), np.square(values(n, "f32", seed + 1)),
                             rng.integers(0, 2 ** 32, n, dtype=np.int64))


def adamw_case(numels, kind, params, views, seed=0):
    """Guarded tensors of a step: end to end in one buffer each, or apart."""
    T = len(numels)
    host = {"g": [values(n, kind, seed + 5 * t) for t, n in enumerate(numels)],
            "w": [values(n, "f32", seed + 5 * t + 1) for t, n in enumerate(numels)]}
    for k, x in zip(("m", "v", "s"), zip(*(moments(n, seed + 5 * t + 2) for t, n in enumerate(numels)))):
        host[k] = list(x)
    kinds = {"g": kind, "w": "f32", "m": "u8", "v": "u8", "s": "u8"}
    if params:
        host["p"], kinds["p"] = [np.zeros(n, f) for n in numels], params
    held, tensors = {}, {}
    for k, arrays in host.items():
        if views:
            held[k] = [Guarded(np.concatenate(arrays), kinds[k], {"s": 2}.get(k, 3))]
            tensors[k] = list(held[k][0].view.split([len(a) for a in arrays]))
        else:
            held[k] = [Guarded(a, kinds[k]) for a in arrays]
            tensors[k] = [x.view for x in held[k]]
    assert len(tensors["g"]) == T
    return host, held, tensors


def host_of(x):
    return x.cpu().numpy() if x.dtype == torch.uint8 else x.float().cpu().numpy()


def assert_weights(got, want, bound, what):
    """Within the bound; where the exact one is not a number the other is not."""
    with np.errstate(all="ignore"):
        got, want = got.astype(np.float64), want.astype(np.float64)
        fine = np.isfinite(want) & np.isfinite(bound)
        off = np.abs(got - want)[fine] - bound[fine]
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert not off.size or off.max() <= 0, f"{what}: {off.max()} past the bound"


def check_adamw8(numels, kind, params, views, step=3, seed=11, norm=None, max_norm=None, on_gpu=False):
    host, held, x = adamw_case(numels, kind, params, views)
    mom = ddp.Moments8(x["m"], x["v"], x["s"])
    t = torch.tensor([step], dtype=torch.int64, device=DEV) if on_gpu else step
    run = ddp.MultiGrad(x["g"]).bind_adamw8(x["w"], mom, params=x.get("p"))
    run(HYPER["lr"], t, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"],
        torch.tensor(norm, device=DEV) if norm is not None else None, max_norm, seed=seed)
    torch.cuda.synchronize()
    c = oracle.clip_factor(norm, max_norm) if norm is not None else f(1)
    for i in range(len(numels)):
        w, m, v, s = mx.adamw8(host["g"][i], host["w"][i], host["m"][i], host["v"][i], host["s"][i], c, *HYPER.values(),
                               step, seed, i)
        assert_weights(host_of(x["w"][i]), w, mx.weight_bound(host["g"][i], host["w"][i], host["m"][i], host["v"][i],
                                                              host["s"][i], c, *HYPER.values(), step), f"w[{i}]")
        assert np.array_equal(host_of(x["s"][i]), s), f"scales[{i}]"
        assert np.array_equal(host_of(x["m"][i]), m), f"m[{i}]"
        assert np.array_equal(host_of(x["v"][i]), v), f"v[{i}]"
        assert_same_bits(host_of(x["g"][i]), host["g"][i], f"g[{i}]")
        if params:
            assert_same_bits(host_of(x["p"][i]), rounded(host_of(x["w"][i]), params), f"params[{i}]")
    for group in held.values():
        for h in group:
            h.intact()


@pytest.mark.parametrize("views", [False, True])
@pytest.mark.parametrize("params", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES)
def test_adamw8(sizes, kind, params, views):
    check_adamw8(SIZES[sizes], kind, params, views, norm=3.0 if views else None, max_norm=1.0 if views else None)


@pytest.mark.parametrize("kind, params, views", [("f32", None, True), ("bf16", "bf16", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("numels", [[700_001, 300_001, 48_574], [700_001, 300_001, 48_575], [1, 1_048_577 + 767, 300, 1057]])
def test_adamw8_long(numels, kind, params, views):
    """2^20 elements in all, for which a wave takes one span, and more, for
    which it takes two."""
    check_adamw8(numels, kind, params, views, on_gpu=views)


@pytest.mark.parametrize("step", [1, 2, 1000, 2 ** 33 + 5])
def test_adamw8_step_numbers(step):
    check_adamw8([700, 33], "bf16", "bf16", False, step=step, on_gpu=False)
    check_adamw8([700, 33], "bf16", "bf16", False, step=step, on_gpu=True, seed=-(2 ** 40) - 3)


def test_adamw8_from_fresh_moments():
    n = 3000
    g = [torch.from_numpy(values(n, "f32", seed=k)).to(DEV) for k in range(4)]
    w = torch.zeros(n, device=DEV)
    mom = ddp.Moments8.zeros(w)
    hw, hm, hv, hs = np.zeros(n, f), np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(2 * 94, np.uint8)
    for t in range(1, 5):
        ddp.adamw8_step(g[t - 1], w, mom, HYPER["lr"], t, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"], seed=5)
        bound = mx.weight_bound(host_of(g[t - 1]), hw, hm, hv, hs, f(1), *HYPER.values(), t)
        hw, hm, hv, hs = mx.adamw8(host_of(g[t - 1]), hw, hm, hv, hs, f(1), *HYPER.values(), t, 5, 0)
        assert_weights(w.cpu().numpy(), hw, bound, f"step {t}")
        hw = w.cpu().numpy()
    assert np.array_equal(host_of(mom.m[0]), hm) and np.array_equal(host_of(mom.v[0]), hv)
    assert np.array_equal(host_of(mom.scales[0]), hs)


def test_adamw8_over_the_exponent_range():
    """Gradients from the least to the largest float32, moments under every
    scale byte: what overflows and what is not a number spreads over its block
    and no further."""
    tops = np.array([m * 2.0 ** k for k in range(-149, 128) for m in (1, 1.75, 1.8751, 1.9375) if m * 2.0 ** k < 3.4e38], f)
    tops = np.concatenate([tops, np.array([np.inf, -np.inf, np.nan], f)])
    x = np.zeros((tops.size, 32), f)
    with np.errstate(all="ignore"):
        for e in range(32):
            x[:, e] = tops * f([1, 0.9, 0.3, -0.1, 0.02, -1, 2.0 ** -9, 2.0 ** -17][e % 8])
    x = x.reshape(-1)
    n = x.size
    rng = np.random.default_rng(0)
    m, v = rng.integers(0, 256, n).astype(np.uint8), rng.integers(0, 256, n).astype(np.uint8)
    m[(m & 127) == 127] = 3
    s = rng.integers(0, 256, 2 * (n // 32)).astype(np.uint8)
    s[1::2] = np.where(s[1::2] < 32, 32, s[1::2])
    g, w = torch.from_numpy(x).to(DEV), torch.zeros(n, device=DEV)
    # a scale byte of m is at most 246 where the step writes it; larger ones decode the same way
    s[0::2] = np.minimum(s[0::2], 246)
    s[0::128] = 255
    mom = ddp.Moments8(*(torch.from_numpy(a).to(DEV) for a in (m, v, s)))
    ddp.adamw8_step(g, w, mom, HYPER["lr"], 2, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"], seed=1)
    bound = mx.weight_bound(x, np.zeros(n, f), m, v, s, f(1), *HYPER.values(), 2)
    hw, hm, hv, hs = mx.adamw8(x, np.zeros(n, f), m, v, s, f(1), *HYPER.values(), 2, 1, 0)
    assert_weights(w.cpu().numpy(), hw, bound, "w")
    assert np.array_equal(host_of(mom.scales[0]), hs)
    assert np.array_equal(host_of(mom.m[0]), hm) and np.array_equal(host_of(mom.v[0]), hv)


@pytest.mark.parametrize("norm", [float("inf"), float("nan")])
def test_adamw8_leaves_a_step_out(norm):
    host, held, x = adamw_case([700, 5], "f32", "bf16", False)
    mom = ddp.Moments8(x["m"], x["v"], x["s"])
    run = ddp.MultiGrad(x["g"]).bind_adamw8(x["w"], mom, params=x["p"])
    run(1e-3, 1, norm=torch.tensor(norm, device=DEV), max_norm=1.0)
    run(1e-3, torch.tensor([0], device=DEV))
    for k in "wmvsp":
        for i in range(2):
            assert np.array_equal(host_of(x[k][i]), host[k][i]), k


def test_adamw8_past_32_bit_offsets():
    """2^30 + 4113 elements: the second piece's random bits, scales and codes."""
    n = 2 ** 30 + 4113
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(n, device=DEV)
    mom = ddp.Moments8.zeros(g)
    places = {at: values(min(4096, n - at), "bf16", seed=k)
              for k, at in enumerate((0, 2 ** 29 + 64, 2 ** 30 - 4096, 2 ** 30, 2 ** 30 + 4096))}
    for at, a in places.items():
        g[at:at + a.size] = torch.from_numpy(a).to(DEV)
    ddp.adamw8_step(g, w, mom, HYPER["lr"], 1, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"], seed=2)
    for at, a in places.items():
        zero = np.zeros(a.size, np.uint8)
        mv, vv = mx.moments_decode(zero, zero, np.zeros(2 * -(-a.size // 32), np.uint8))
        hw, mv, vv = oracle.adamw(a, np.zeros(a.size, f), mv, vv, f(1), *HYPER.values(), 1)
        m, v, s = mx.moments_encode(mv, vv, mx.random_bits(a.size, 2, 1, 0, first=at))
        bound = mx.weight_bound(a, np.zeros(a.size, f), zero, zero, np.zeros(2 * -(-a.size // 32), np.uint8), f(1),
                                *HYPER.values(), 1)
        assert_weights(host_of(w[at:at + a.size]), hw, bound, f"w at {at}")
        assert np.array_equal(host_of(mom.m[0][at:at + a.size]), m), at
        assert np.array_equal(host_of(mom.v[0][at:at + a.size]), v), at
        assert np.array_equal(host_of(mom.scales[0][at // 16:at // 16 + s.size]), s), at


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES)
def test_read_moments(sizes, kind):
    numels = SIZES[sizes]
    codes = [moments(n, 7 * t) for t, n in enumerate(numels)]
    held = [Guarded(np.concatenate(x), "u8", o) for x, o in zip(zip(*codes), (1, 3, 2))]
    mom = ddp.Moments8(held[0].view.split(numels), held[1].view.split(numels),
                       held[2].view.split([c[2].size for c in codes]))
    out = [Guarded(np.zeros(sum(numels), f), kind, 5) for _ in range(2)]
    mom.bind_read(*(o.view.split(numels) for o in out))()
    torch.cuda.synchronize()
    new = mom.read(torch_dtype(kind))
    for t, (m, v, s) in enumerate(codes):
        for which, want in enumerate(mx.moments_decode(m, v, s)):
            assert_same_bits(host_of(out[which].view.split(numels)[t]), rounded(want, kind), f"{which} of {t}")
            assert_same_bits(host_of(new[which][t]), rounded(want, kind), f"{which} of {t}")
    for h in held + out:
        h.intact()


def test_read_every_code():
    m = np.repeat(np.arange(256, dtype=np.uint8), 256)
    v = np.tile(np.arange(256, dtype=np.uint8), 256)
    for sm, sv in ((0, 0), (1, 32), (127, 127), (246, 254), (255, 255), (30, 200)):
        s = np.tile(np.array([sm, sv], np.uint8), m.size // 32)
        a = np.zeros_like(m) if sm == 0 else m
        a = np.full_like(m, 127) if sm == 255 else a
        got = ddp.Moments8(*(torch.from_numpy(x).to(DEV) for x in (a, v, s))).read()
        for x, want in zip(got, mx.moments_decode(a, v, s)):
            assert_same_bits(x[0].cpu().numpy(), want, f"scales {sm} {sv}")


# ------------------------------------------------------- the step whole ----

def host_step(state, grads, P, n, lr, t):
    """One step on the host: quantise with residual, all-reduce with norm,
    clipped AdamW."""
    rows = []
    for r in range(P):
        codes, scales, state["left"][r] = mx.mx4_quantize(grads[r], state["left"][r])
        state["left"][r] = rounded(state["left"][r], "bf16")
        rows.append(mx.mx4_decode(codes, scales, n))
    g = mx.mx4_allreduce(np.stack(rows), "mean")
    return g, f(np.sqrt(np.square(g.astype(np.float64)).sum()))


def test_steps_of_a_job():
    P, n, steps = 4, 9001, 5
    plan = ddp.GradBucketer([(n,)], torch.bfloat16, 1 << 12)
    arena = plan.alloc_arena(P)
    rows = [arena[r, :n] for r in range(P)]
    left = plan.alloc_arena(P).zero_()
    left = [left[r, :n] for r in range(P)]
    coded = plan.alloc_mx4(P)
    grad, w = torch.empty(n, device=DEV), plan.alloc_state(1)[0]
    params = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    w.copy_(torch.from_numpy(values(n, "f32", seed=99)))
    mom = ddp.Moments8.zeros(grad)
    step = ddp.MultiGrad(grad).bind_adamw8(w, mom, params=params)
    state = {"left": [np.zeros(n, f) for _ in range(P)]}
    hw, hm, hv, hs = w.cpu().numpy(), np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(2 * -(-n // 32), np.uint8)
    for t in range(1, steps + 1):
        grads = [values(n, "bf16", seed=10 * t + r) for r in range(P)]
        for r in range(P):
            rows[r].copy_(torch.from_numpy(grads[r]))
        ddp.mx4_quantize(rows, residual=left, out=coded)
        _, norm = ddp.allreduce_mx4_norm(coded, "mean", out=[grad])
        step(1e-3, t, (0.9, 0.99), 1e-8, 0.1, norm=norm, max_norm=1.0, seed=3)
        g, want_norm = host_step(state, grads, P, n, 1e-3, t)
        assert_same_bits(grad.cpu().numpy(), g, f"step {t}")
        assert float(norm) == pytest.approx(float(want_norm), rel=2.0 ** -23)
        c = oracle.clip_factor(float(norm), 1.0)
        bound = mx.weight_bound(g, hw, hm, hv, hs, c, 1e-3, 0.9, 0.99, 1e-8, 0.1, t)
        hw, hm, hv, hs = mx.adamw8(g, hw, hm, hv, hs, c, 1e-3, 0.9, 0.99, 1e-8, 0.1, t, 3, 0)
        assert_weights(w.cpu().numpy(), hw, bound, f"step {t}")
        hw = w.cpu().numpy()
    assert_same_bits(params.float().cpu().numpy(), rounded(hw, "bf16"))
    assert np.array_equal(host_of(mom.m[0]), hm) and np.array_equal(host_of(mom.v[0]), hv)
    for r in range(P):
        assert_same_bits(left[r].float().cpu().numpy(), state["left"][r])


def job(n, P, seed):
    rows = [torch.from_numpy(values(n, "bf16", seed=seed + r)).to(DEV).bfloat16() for r in range(P)]
    x = {"rows": rows, "left": [torch.zeros(n, device=DEV) for _ in range(P)],
         "coded": [ddp.Mx4.empty(n, DEV) for _ in range(P)], "grad": torch.zeros(n, device=DEV),
         "again": ddp.Mx4.empty(n, DEV), "owner": torch.zeros(n, device=DEV),
         "w": torch.ones(n, device=DEV), "count": torch.zeros(1, dtype=torch.int64, device=DEV),
         "read": [torch.zeros(n, device=DEV) for _ in range(2)]}
    x["moments"] = ddp.Moments8.zeros(x["grad"])
    step = ddp.MultiGrad(x["grad"]).bind_adamw8(x["w"], x["moments"])
    read = x["moments"].bind_read(*x["read"])

    def once():
        x["count"] += 1
        ddp.mx4_quantize(x["rows"], residual=x["left"], out=x["coded"])
        ddp.allreduce_mx4(x["coded"], "mean", out=[x["again"]], residual=x["owner"])
        _, x["norm"] = ddp.allreduce_mx4_norm(x["coded"], "mean", out=[x["grad"]])
        step(1e-3, x["count"], norm=x["norm"], max_norm=1.0, seed=4)
        read()
    return x, once


def job_state(x):
    return [t.clone() for t in (*x["left"], *(c.codes for c in x["coded"]), x["again"].codes, x["owner"], x["grad"],
                                x["w"], *x["moments"].m, *x["moments"].v, *x["moments"].scales, *x["read"], x["norm"])]


@pytest.mark.parametrize("n", [3001, 3_000_001])
def test_graphs_replayed_between_eager_calls(n):
    a, eager = job(n, 3, 0)
    b, captured = job(n, 3, 0)
    c, other = job(n, 3, 50)
    captured(), eager()                       # one step before the capture, on both sides
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            captured()
    torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        other()
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(job_state(a), job_state(b))):
            assert torch.equal(p, q), (k, i)


def test_two_jobs_on_two_streams():
    n = 2_000_003
    wanted = []
    for seed in (0, 70):
        x, once = job(n, 4, seed)
        for _ in range(3):
            once()
        torch.cuda.synchronize()
        wanted.append(job_state(x))
    jobs = [job(n, 4, seed) for seed in (0, 70)]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (_, once), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                once()
    torch.cuda.synchronize()
    for (x, _), want in zip(jobs, wanted):
        assert all(torch.equal(p, q) for p, q in zip(job_state(x), want))


def test_two_graphs_replayed_in_turn():
    """Two captured jobs share neither workspace nor scratch memory: replayed in
    turn and on two streams, each goes on as its eager twin does."""
    n = 1_000_003
    twins = [job(n, 3, seed) for seed in (0, 40)]
    jobs = [job(n, 3, seed) for seed in (0, 40)]
    for _, once in twins + jobs:
        once()
    graphs = []
    for _, once in jobs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                once()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append((graph, side))
    for k in range(3):
        for (graph, side), (_, eager) in zip(graphs, twins):
            if k == 1:
                graph.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    graph.replay()
            eager()
        torch.cuda.synchronize()
        for (a, _), (b, _) in zip(twins, jobs):
            for i, (p, q) in enumerate(zip(job_state(a), job_state(b))):
                assert torch.equal(p, q), (k, i)


def test_with_another_gpu_current(monkeypatch):
    """A call that finds another GPU current makes the tensors' one current for
    its launches (seen from one GPU: the first question is answered wrongly, the
    results are the same)."""
    n = 5000
    a, once = job(n, 2, 0)
    once()
    x, _ = job(n, 2, 0)
    real, wrong = torch.cuda.current_device, []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: wrong.pop() if wrong else real())
    step = ddp.MultiGrad(x["grad"]).bind_adamw8(x["w"], x["moments"])
    read = x["moments"].bind_read(*x["read"])
    x["count"] += 1
    calls = [lambda: ddp.mx4_quantize(x["rows"], residual=x["left"], out=x["coded"]),
             lambda: ddp.allreduce_mx4(x["coded"], "mean", out=[x["again"]], residual=x["owner"]),
             lambda: x.update(norm=ddp.allreduce_mx4_norm(x["coded"], "mean", out=[x["grad"]])[1]),
             lambda: step(1e-3, x["count"], norm=x["norm"], max_norm=1.0, seed=4), read,
             lambda: x.update(values=ddp.mx4_dequantize(x["coded"]))]
    for call in calls:
        wrong.append(real() + 1)
        call()
        assert not wrong
    monkeypatch.undo()
    assert all(torch.equal(p, q) for p, q in zip(job_state(a), job_state(x)))
    assert torch.equal(x["values"][1], ddp.mx4_dequantize(a["coded"])[1])


def test_moments_read_back_go_on_in_32_bits():
    """The 8-bit step's weights are those of the 32-bit step on the moments read
    back before it."""
    numels = [3000, 41]
    host, _, x = adamw_case(numels, "f32", None, False)
    mom = ddp.Moments8(x["m"], x["v"], x["s"])
    m, v = mom.read()
    w = [t.clone() for t in x["w"]]
    ddp.adamw_step(x["g"], w, m, v, 1e-2, 7, (0.9, 0.99), 1e-8, 0.1)
    ddp.adamw8_step(x["g"], x["w"], mom, 1e-2, 7, (0.9, 0.99), 1e-8, 0.1, seed=1)
    for i in range(2):
        bound = mx.weight_bound(host["g"][i], host["w"][i], host["m"][i], host["v"][i], host["s"][i], f(1),
                                *HYPER.values(), 7)
        assert_weights(host_of(x["w"][i]), host_of(w[i]), bound, f"w[{i}]")
        # the codes lie next to the 32-bit moments: within one step of a code, 1/8 of
        # the value or of the least code's distance
        for got, want, least in ((mom.read()[0][i], m[i], 2.0 ** -9), (mom.read()[1][i], v[i], 2.0 ** -31)):
            scale = np.repeat(host_of(mom.scales[i]).reshape(-1, 2)[:, 0 if want is m[i] else 1].astype(float), 32)
            scale = 2.0 ** (scale[:numels[i]] - 127)
            d = np.abs(host_of(got).astype(np.float64) - host_of(want))
            assert (d <= np.maximum(np.abs(host_of(want)) / 8 * (1 + 2.0 ** -20), least * scale * 1.0001)).all()


def test_same_call_same_bits():
    n = 300_007
    a, first = job(n, 4, 0)
    b, second = job(n, 4, 0)
    for _ in range(3):
        first(), second()
    assert all(torch.equal(p, q) for p, q in zip(job_state(a), job_state(b)))
    # another seed rounds otherwise
    g = torch.ones(n, device=DEV)
    states = [ddp.Moments8.zeros(g) for _ in range(2)]
    for seed, mom in enumerate(states):
        ddp.adamw8_step(g * 0.3, torch.zeros(n, device=DEV), mom, 1e-3, 1, (0.9, 0.99), seed=seed)
    share = (states[0].m[0] != states[1].m[0]).float().mean()
    # m = 0.03 lies between 0.0293 (15 * 2^-9) and 0.03125: up with p = 0.36, so two seeds differ at
    # 2 p (1 - p) = 0.46 of the elements; deviation 0.5 / sqrt(n) = 0.0009, five of those
    p = float((f(0.1) * f(0.3)) * 512 - 15)
    assert abs(float(share) - 2 * p * (1 - p)) < 0.0046


@pytest.mark.parametrize("count", [139, 140, 160, 161, 162, 163, 164, 165, 323, 325])
@pytest.mark.parametrize("params", [None, "bf16"])
def test_adamw8_at_the_launches_limits(count, params):
    """As many tensors as a launch holds, and one more; every fifth empty, the
    last two as well, so that launches end and begin with empty ones."""
    numels = [0 if t % 5 == 4 or t >= count - 2 else 1 + 53 * t % 300 for t in range(count)]
    check_adamw8(numels, "f32", params, True)
    codes = [moments(n, t) for t, n in enumerate(numels)]
    held = [torch.from_numpy(np.concatenate(x)).to(DEV) for x in zip(*codes)]
    mom = ddp.Moments8(held[0].split(numels), held[1].split(numels), held[2].split([c[2].size for c in codes]))
    new = mom.read()
    for t, c in enumerate(codes):
        for which, want in enumerate(mx.moments_decode(*c)):
            assert_same_bits(host_of(new[which][t]), want, f"{which} of {t}")


def test_adamw8_long_tensor_among_short_ones():
    """A tensor of two pieces has launches of its own, and the tensors around it
    keep their numbers in the call; its values read back past 2^30 too."""
    numels = [33, 2 ** 30 + 777, 0, 700]
    g = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in numels]
    w = [torch.zeros(n, device=DEV) for n in numels]
    mom = ddp.Moments8.zeros(g)
    places = {(0, 0): values(33, "bf16", 1), (1, 0): values(640, "bf16", 2), (1, 2 ** 30 - 64): values(64, "bf16", 3),
              (1, 2 ** 30): values(777, "bf16", 4), (3, 0): values(700, "bf16", 5)}
    for (t, at), a in places.items():
        g[t][at:at + a.size] = torch.from_numpy(a).to(DEV)
    ddp.adamw8_step(g, w, mom, HYPER["lr"], 1, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"], seed=8)
    read = mom.read(torch.bfloat16)
    for (t, at), a in places.items():
        zero = np.zeros(a.size, np.uint8)
        _, mv, vv = oracle.adamw(a, np.zeros(a.size, f), zero.astype(f), zero.astype(f), f(1), *HYPER.values(), 1)
        m, v, s = mx.moments_encode(mv, vv, mx.random_bits(a.size, 8, 1, t, first=at))
        got_s = host_of(mom.scales[t][at // 16:at // 16 + s.size])
        assert np.array_equal(got_s, s) and np.array_equal(host_of(mom.m[t][at:at + a.size]), m), (t, at)
        assert np.array_equal(host_of(mom.v[t][at:at + a.size]), v), (t, at)
        for which, want in enumerate(mx.moments_decode(m, v, s)):
            assert_same_bits(host_of(read[which][t][at:at + a.size]), rounded(want, "bf16"), f"{which} of {t} at {at}")


@pytest.mark.parametrize("params, norm", [(None, None), ("bf16", 3.0)])
@pytest.mark.parametrize("kind, nan", [("bf16", 0xFFFF0000), ("bf16", 0xFF810000), ("bf16", 0x7FFF0000),
                                       ("f32", 0xFFFFFFFF), ("f32", 0xFFF00001), ("f32", 0xFF800001), ("f32", 0x7FFFFFFF)])
def test_adamw8_of_any_nan(kind, nan, params, norm):
    """A NaN of either sign and any payload: its block of m NaN, of v infinite,
    the other blocks as without it; in whole spans and in a tensor's end."""
    n, places = 2048 + 70, (5, 1000, 2047, 2100)
    g = values(n, kind, seed=1)
    g.view(np.uint32)[list(places)] = nan
    w, (m, v, s) = values(n, "f32", seed=2), moments(n, 3)
    bits16 = torch.from_numpy((g.view(np.uint32) >> 16).astype(np.uint16).view(np.int16))
    grad = (bits16.view(torch.bfloat16) if kind == "bf16" else torch.from_numpy(g)).to(DEV)
    mom = ddp.Moments8(*(torch.from_numpy(x).to(DEV) for x in (m, v, s)))
    weights = torch.from_numpy(w.copy()).to(DEV)
    out = torch.zeros(n, dtype=torch_dtype(params), device=DEV) if params else None
    ddp.adamw8_step(grad, weights, mom, HYPER["lr"], 3, (HYPER["b1"], HYPER["b2"]), HYPER["eps"], HYPER["wd"], params=out,
                    norm=torch.tensor(norm, device=DEV) if norm else None, max_norm=1.0 if norm else None, seed=6)
    c = oracle.clip_factor(norm, 1.0) if norm else f(1)
    bound = mx.weight_bound(g, w, m, v, s, c, *HYPER.values(), 3)
    hw, hm, hv, hs = mx.adamw8(g, w, m, v, s, c, *HYPER.values(), 3, 6, 0)
    assert (hs[[2 * (at // 32) + 1 for at in places]] == 255).all() and (hs == 255).sum() == 2 * len(places)
    assert np.array_equal(host_of(mom.scales[0]), hs)
    assert np.array_equal(host_of(mom.m[0]), hm) and np.array_equal(host_of(mom.v[0]), hv)
    assert_weights(weights.cpu().numpy(), hw, bound, "w")
    assert np.isnan(hw).sum() == len(places)
