"""The Python handles of the gradient norm, clipping and AdamW calls on the
host: what they keep alive, and which memory they pass on.  CPU tensors stand
in for GPU ones and a stub for the library's launching calls."""

import gc
import weakref

import pytest
import torch

ddp = pytest.importorskip("gradient_all_reduce_allreduce_amd")
from gradient_all_reduce_allreduce_amd import _native as N  # noqa: E402
from gradient_all_reduce_allreduce_amd import api  # noqa: E402

LAUNCHING = ("grad_norm_multi", "grad_clip_multi", "adamw_step_multi")


class Gpu(torch.Tensor):
    """A CPU tensor that says it lives on the GPU."""
    is_cuda = True


def gpu(n, dtype=torch.float32):
    return torch.Tensor._make_subclass(Gpu, torch.zeros(n, dtype=dtype))


class Lib:
    """The library with its launching calls written down instead of made."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in LAUNCHING:
            return lambda *args: self.calls.append((name, args)) or N.DDP_OK
        return getattr(self.real, name)


@pytest.fixture
def lib(monkeypatch):
    stub = Lib(N.lib())
    monkeypatch.setattr(N, "lib", lambda: stub)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)    # a CPU tensor's device index
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    return stub


CALLS = {
    "norm": lambda g, s: ddp.grad_norm(g),
    "clip": lambda g, s: ddp.clip_grads(g, 1.0),
    "clip_into": lambda g, s: ddp.clip_grads(g, 1.0, out=s[0]),
    "adamw": lambda g, s: ddp.adamw_step(g, *s[:3], 1e-3, 1, params=s[3]),
    "bound_clip": lambda g, s: ddp.MultiGrad(g).bind_clip(s[0])(1.0),
    "bound_adamw": lambda g, s: ddp.MultiGrad(g).bind_adamw(*s[:3], params=s[3])(1e-3, 1),
}


@pytest.mark.parametrize("call", CALLS)
def test_nothing_outlives_a_call(lib, call):
    """Gradients made anew at each step are freed as soon as the last
    reference goes, without the cyclic collector."""
    grads = [gpu(100), gpu(7)]
    state = [[gpu(100), gpu(7)] for _ in range(4)]
    refs = [weakref.ref(t) for t in grads + sum(state, [])]
    gc.collect()
    gc.disable()
    try:
        CALLS[call](grads, state)
        assert len(lib.calls) == 1
        lib.calls.clear()
        del grads, state
        assert not any(r() is not None for r in refs)
    finally:
        gc.enable()


def test_a_bound_call_keeps_its_tensors(lib):
    """While the bound call lives, so do the tensors whose addresses it
    holds."""
    grads, state = [gpu(100)], [[gpu(100)] for _ in range(4)]
    refs = [weakref.ref(t) for t in grads + sum(state, [])]
    mg = ddp.MultiGrad(grads)
    clip, step = mg.bind_clip(state[3]), mg.bind_adamw(*state[:3])
    del mg, grads, state
    gc.collect()
    assert all(r() is not None for r in refs)
    clip(1.0)
    step(1e-3, 1)
    assert [name for name, _ in lib.calls] == ["grad_clip_multi", "adamw_step_multi"]


def swap_data(t):
    t.data = gpu(t.numel(), t.dtype)


def swap_storage(t):
    t.set_(gpu(t.numel(), t.dtype))


MOVES = {
    "data": swap_data,
    "set": swap_storage,
    "grown": lambda t: t.resize_(100_000),
    "shrunk": lambda t: t.resize_(3),
    "freed": lambda t: t.untyped_storage().resize_(0),
}


@pytest.mark.parametrize("move", MOVES)
@pytest.mark.parametrize("which", ["grads", "out", "w", "m", "v", "params"])
def test_a_tensor_given_other_memory_is_refused(lib, which, move):
    """A held tensor that lies elsewhere, or has another size, than when it
    was bound: its old address may be anyone's."""
    t = {k: [gpu(100), gpu(64)] for k in ("grads", "out", "w", "m", "v", "params")}
    mg = ddp.MultiGrad(t["grads"])
    clip, step = mg.bind_clip(t["out"]), mg.bind_adamw(t["w"], t["m"], t["v"], t["params"])
    calls = {"norm": mg.norm, "clip": lambda: clip(1.0), "adamw": lambda: step(1e-3, 1)}
    reads = {"grads": ("norm", "clip", "adamw"), "out": ("clip",)}.get(which, ("adamw",))
    for call in calls.values():
        call()
    lib.calls.clear()
    MOVES[move](t[which][1])
    for name, call in calls.items():
        if name in reads:
            with pytest.raises(ValueError, match=rf"{which}\[1\]"):
                call()
        else:
            call()
    assert len(lib.calls) == 3 - len(reads)


def test_in_place_clip_of_a_tensor_given_other_memory(lib):
    grads = [gpu(100), gpu(64)]
    clip = ddp.MultiGrad(grads).bind_clip()
    swap_data(grads[0])
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        clip(1.0)
    assert not lib.calls


def test_values_and_flags_may_change(lib):
    """What moves no memory is no reason to refuse."""
    g = gpu(100)
    mg = ddp.MultiGrad([g])
    g.fill_(3.0)
    g.requires_grad_(True)
    mg.norm()
    mg.bind_clip()(1.0)
    assert len(lib.calls) == 2


def test_memory_is_held_with_its_tensor(lib):
    """The memory that a bound tensor was taken away from is not handed to
    another while the handle holds its address."""
    from torch.multiprocessing.reductions import StorageWeakRef
    g, out = gpu(100), gpu(100)
    old = [StorageWeakRef(t.untyped_storage()) for t in (g, out)]
    mg = ddp.MultiGrad([g])
    clip = mg.bind_clip([out])
    swap_data(g)
    swap_data(out)
    assert not any(s.expired() for s in old)
    del mg, clip
    assert all(s.expired() for s in old)


def test_tensors_without_elements_are_held_too(lib):
    g = [gpu(0), gpu(5)]
    mg = ddp.MultiGrad(g)
    mg.norm()
    g[0].resize_(8)
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        mg.norm()
    assert len(lib.calls) == 1


def addresses(array, count):
    return [array[k] for k in range(count)]


def test_parameters_without_a_gradient_are_skipped(lib):
    """grad_norm and clip_grads of [p.grad for p in model.parameters()], where
    a frozen or unused parameter's is None."""
    a, b = gpu(100), gpu(7)
    ddp.grad_norm([None, a, None, b])
    ddp.clip_grads((x for x in (a, None, b)), 1.0)
    x, y = gpu(100), gpu(7)
    ddp.clip_grads([a, None, b], 1.0, out=[x, None, y])
    ddp.clip_grads([a, None, b], 1.0, out=[x, gpu(9), y])       # the place of a skipped one
    want = [a.data_ptr(), b.data_ptr()]
    outs = [want] + 2 * [[x.data_ptr(), y.data_ptr()]]
    assert [name for name, _ in lib.calls] == ["grad_norm_multi"] + 3 * ["grad_clip_multi"]
    for k, (_, args) in enumerate(lib.calls):
        assert args[0] == 2 and addresses(args[1], 2) == [100, 7] and addresses(args[2], 2) == want
        if k:
            assert addresses(args[4], 2) == outs[k - 1]


def test_skipping_refusals(lib):
    a = gpu(5)
    for call in (lambda: ddp.grad_norm([None]), lambda: ddp.clip_grads([None, None], 1.0),
                 lambda: ddp.clip_grads([a, None], 1.0, out=[gpu(5)]),
                 lambda: ddp.clip_grads([a, None], 1.0, out=[None, gpu(5)])):
        with pytest.raises((ValueError, TypeError)):
            call()
    # one tensor per entry where every entry has a state of its own
    for call in (lambda: ddp.MultiGrad([a, None]), lambda: ddp.MultiGrad([None, a]),
                 lambda: ddp.adamw_step([a, None], [a, a], [a, a], [a, a], 1e-3, 1),
                 lambda: ddp.adamw_step([a], [None], [a], [a], 1e-3, 1), lambda: ddp.grad_norm([a, 3.0])):
        with pytest.raises(TypeError, match="tensor"):
            call()
    assert not lib.calls
