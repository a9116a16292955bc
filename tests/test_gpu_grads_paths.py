"""The norm, clipping and all-reduce with norm at the sizes where their code
changes path: tile ends of the many-workgroup kernels, the last set that one
workgroup takes and the first that it does not, and a bucketed all-reduce whose
partial sums have a second level.  Each test asserts which path it takes.
Tolerances as in test_gpu_grads.py: the norm within one rounding of float64,
everything else bit for bit."""

import gc

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import DEV, assert_same_bits, oracle_ring, to_device, to_host, torch_dtype
from test_gpu_grads import SIZES, Arena, check_norm, clipped, draw, rank_draw, same, separate

pytestmark = pytest.mark.gpu
ddp = pytest.importorskip("gradient_all_reduce_allreduce_amd")

ES = {"f32": 4, "bf16": 2}
SMALL = 4096                      # bytes of a piece of the one-workgroup path, and of a clip tile
WIDE = 16384                      # bytes of a norm tile
PIECES = 64                       # that one workgroup takes


def takes_one_workgroup(tensors):
    codes = [ddp.BF16 if t.dtype == torch.bfloat16 else ddp.F32 for t in tensors]
    need = ddp.grad_norm_workspace_bytes([t.numel() for t in tensors], [t.data_ptr() for t in tensors], codes)
    assert need in (0, ddp.NORM_WORKSPACE_BYTES)
    return need == 0


class Placed(Arena):
    """As Arena, every tensor `off` elements past a line."""

    def __init__(self, arrays, types, off):
        place, used = [], dict.fromkeys(types, 0)
        for a, k in zip(arrays, types):
            place.append(used[k] + off)
            used[k] += (off + len(a)) // 64 * 64 + 128
        self.held, self.views, self.at = {}, [], []
        for k, total in used.items():
            x = torch.full((total * ES[k],), self.CANARY, dtype=torch.uint8, device=DEV)
            self.held[k] = x.view(torch_dtype(k))
            assert x.data_ptr() % 128 == 0
        for a, k, o in zip(arrays, types, place):
            v = self.held[k][o:o + len(a)]
            v.copy_(torch.from_numpy(a))
            self.views.append(v)
            self.at.append((k, o, len(a)))


def check_norm_and_clip(arrays, types, place, one_workgroup):
    """Norm; clip with its own norm into other tensors and in place."""
    src = place(arrays, types)
    dst = place([np.zeros_like(a) for a in arrays], types)
    assert takes_one_workgroup(src.views) == one_workgroup
    norm = ddp.grad_norm(src.views)
    check_norm(norm, arrays)
    limit = 0.5 * oracle.grad_norm(arrays)
    want = clipped(arrays, types, np.float32(float(norm)), limit)
    assert torch.equal(ddp.clip_grads(src.views, limit, out=dst.views), norm)
    same(dst.host(), want, "out")
    same(src.host(), arrays, "inputs")
    dst.check_canaries()
    assert torch.equal(ddp.clip_grads(src.views, limit), norm)
    same(src.host(), want, "in place")
    src.check_canaries()


@pytest.mark.parametrize("off", [0, 1, 31])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_path_at_tile_ends(dtype, off):
    """Tensors that end one element before, at and one past the end of a tile,
    of the norm's and of the clip's, each beginning on a line or `off`
    elements past it."""
    sizes = []
    for tile in (SMALL // ES[dtype], WIDE // ES[dtype]):
        sizes += [k * tile - off + d for k in (1, 2, 3) for d in (-1, 0, 1)]
    arrays, types = draw(sizes, dtype, seed=off)
    check_norm_and_clip(arrays, types, lambda a, t: Placed(a, t, off), one_workgroup=False)


@pytest.mark.parametrize("off", [0, 5])
def test_wide_path_at_tile_ends_of_both_types(off):
    sizes = [k * WIDE // es - off + d for k in (1, 2) for d in (-1, 0, 1) for es in (2, 4)]     # "mixed" begins with bf16
    arrays, types = draw(sizes, "mixed", seed=7 + off)
    check_norm_and_clip(arrays, types, lambda a, t: Placed(a, t, off), one_workgroup=False)


def pieces(kind, dtype):
    """Sets of exactly 64 pieces when every tensor begins on a line."""
    count = {"one": 1, "single": PIECES, "full": PIECES, "rest": PIECES // 2, "last": PIECES - 1}[kind]
    es = [ES[("bf16", "f32")[t % 2] if dtype == "mixed" else dtype] for t in range(count)]
    if kind == "one":
        return [PIECES * SMALL // es[0]]
    if kind == "last":
        return [3] * (count - 1) + [2 * SMALL // es[-1] - 1]
    return [{"single": 1, "full": SMALL // e, "rest": SMALL // e + 1}[kind] for e in es]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("kind", ["one", "single", "full", "rest", "last"])
@pytest.mark.parametrize("more", [False, True])
def test_at_the_limit_of_the_one_workgroup_path(kind, dtype, more):
    """64 pieces fill the last slots of that path's arguments and registers;
    one more goes to the wide kernels."""
    arrays, types = draw(pieces(kind, dtype) + [1] * more, dtype, seed=len(kind))
    check_norm_and_clip(arrays, types, lambda a, t: Placed(a, t, 0), one_workgroup=not more)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_limit_of_a_tensor_off_a_line(dtype):
    """One tensor whose lead makes up for its end: 64 pieces, and 65."""
    n = PIECES * SMALL // ES[dtype]
    for count in (n - 3, n - 2):
        arrays, types = draw([count], dtype, seed=count)
        check_norm_and_clip(arrays, types, lambda a, t: Placed(a, t, 3), one_workgroup=count == n - 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES)
def test_clip_in_place_with_its_own_norm(sizes, dtype):
    """What a training loop does, for separate tensors: few and many, of both
    types, over several launches."""
    arrays, types = draw(SIZES[sizes], dtype)
    limit = 0.5 * oracle.grad_norm(arrays)
    ts = separate(arrays, types)
    norm = ddp.clip_grads(ts, limit)
    check_norm(norm, arrays)
    same([t.float().cpu().numpy() for t in ts], clipped(arrays, types, np.float32(float(norm)), limit))


@pytest.mark.parametrize("pair", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("copies", ["ranks", "one"])
@pytest.mark.parametrize("C,E,n,launches", [(8, 262_144, 9 * 262_144 + 4_444, 1),
                                            (8, 250_008, 9 * 250_008 + 12_345, 2),
                                            (16, 250_008, 9 * 250_008 + 12_345, 10)])
def test_allreduce_norm_buckets_of_many_partials(C, E, n, launches, copies, pair):
    """Over 4,096 workgroups, the full buckets and the tail as one ring, as one
    each, and every bucket as its own: the partial sums
    of every launch lie behind each other, and every launch clears the count
    that their sum starts from.  Two calls in a row whose workspace, taken from
    torch's allocator, begins as ones and as the call before left it."""
    it, ot = pair
    P = 8
    codes = [ddp.BF16 if k == "bf16" else ddp.F32 for k in pair]
    need = ddp.allreduce_norm_workspace_bytes(P, C, *codes, n, E)
    assert need > 8 * 4096
    assert ddp.ddp_buckets_launch_count(P, C, *codes, False, n, E) == launches
    X = [rank_draw(P, n, it, seed=k) for k in (1, 2)]
    ins = [to_device(x, it) for x in X]
    out = [[torch.empty(n, dtype=torch_dtype(ot), device=DEV) for _ in range(P if copies == "ranks" else 1)]
           for _ in X]
    torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)           # freed at once: the next of its size
    norms = [ddp.allreduce_norm(i, "mean", C, out=o, bucket_elems=E)[1] for i, o in zip(ins, out)]
    for x, o, norm in zip(X, out, norms):
        want = np.concatenate([oracle_ring(x[:, lo:lo + E], "mean", C, in_dtype=it, out_dtype=ot)
                               for lo in range(0, n, E)], axis=1)
        assert_same_bits(to_host(o), want[:len(o)], "outputs")
        check_norm(norm, [oracle.bf16_bits_to_f32(want[0]) if ot == "bf16" else want[0]])


# ---------------------------------------------------------------- handles ----

def test_gradients_made_anew_are_freed_without_the_collector():
    n = 1 << 20
    state = [[torch.zeros(n, device=DEV)] for _ in range(3)]

    def step(k):
        g = [torch.ones(n, device=DEV)]
        ddp.clip_grads(g, 1.0)
        ddp.adamw_step(g, *state, 1e-3, k)
    step(1)
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        for k in range(2, 12):
            step(k)
        assert torch.cuda.memory_allocated() == before
    finally:
        gc.enable()


def test_moved_memory_is_refused_and_left_alone():
    g = [torch.full((5000,), 2.0, device=DEV), torch.full((64,), 2.0, device=DEV)]
    mg = ddp.MultiGrad(g)
    clip = mg.bind_clip()
    old = g[1].detach()
    g[1].data = torch.full((64,), 2.0, device=DEV)
    for call in (mg.norm, lambda: clip(1.0)):
        with pytest.raises(ValueError, match=r"grads\[1\]"):
            call()
    assert all(bool((x == 2).all()) for x in g + [old])
    norm = ddp.clip_grads(g, 1.0)
    check_norm(norm, [np.full(5064, 2.0, np.float32)])


def test_entries_without_a_gradient():
    arrays, types = draw([3000, 17], "f32", 0.1)
    a, b = separate(arrays, types)
    norm = ddp.grad_norm([None, a, None, b])
    check_norm(norm, arrays)
    out = [torch.empty_like(a), None, torch.empty_like(b)]
    assert torch.equal(ddp.clip_grads([a, None, b], 0.5, out=out), norm)
    same([out[0].cpu().numpy(), out[2].cpu().numpy()], clipped(arrays, types, np.float32(float(norm)), 0.5))
