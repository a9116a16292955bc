"""Refusals of the 4-bit gradient and 8-bit moment calls: host only, every
call returns before any launch."""

import ctypes

import pytest
import torch

ddp = pytest.importorskip("gradient_all_reduce_allreduce_amd")
from gradient_all_reduce_allreduce_amd import _native as N  # noqa: E402
from gradient_all_reduce_allreduce_amd.api import DdpError  # noqa: E402

BASE = 0x7f0000000000          # never dereferenced
STEP = 1 << 20
WS, NORM, STEPS = BASE + (1 << 36), BASE + (1 << 37), BASE + (1 << 38)
NAN, INF = float("nan"), float("inf")


def at(k, off=0):
    return BASE + k * STEP + off


def refused(fn, args, status, text=None):
    with pytest.raises(DdpError) as e:
        fn(**args)
    assert e.value.status == status, e.value
    if text:
        assert text in str(e.value)


def quantize_args(**change):
    a = dict(P=2, rank_in=[at(0), at(1)], in_dtype=ddp.F32, n=1000, rank_residual=[at(2), at(3)], residual_dtype=ddp.BF16,
             rank_codes=[at(4), at(5)], rank_scales=[at(6), at(7)])
    a.update(change)
    return a


def dequantize_args(**change):
    a = dict(P=2, rank_codes=[at(4), at(5)], rank_scales=[at(6), at(7)], n=1000, rank_out=[at(0), at(1)], out_dtype=ddp.F32)
    a.update(change)
    return a


def reduce_args(**change):
    a = dict(op="mean", P=2, rank_codes=[at(4), at(5)], rank_scales=[at(6), at(7)], n=1000, rank_out=[at(0), at(1)],
             out_dtype=ddp.F32, norm=NORM, workspace=WS, workspace_bytes=8)
    a.update(change)
    return a


def coded_args(**change):
    a = dict(op="mean", P=2, rank_codes=[at(4), at(5)], rank_scales=[at(6), at(7)], n=1000, out_codes=[at(8), at(9)],
             out_scales=[at(10), at(11)], residual=at(2), residual_dtype=ddp.F32, norm=NORM, workspace=WS,
             workspace_bytes=8)
    a.update(change)
    return a


def adamw_args(**change):
    a = dict(numels=[100, 0, 7], grads=[at(0), 0, at(2)], grad_dtype=ddp.BF16, w=[at(3), 0, at(4)],
             m=[at(5, 1), 0, at(6)], v=[at(7), 0, at(8, 3)], scales=[at(11, 2), 0, at(12)], params=[at(9), 0, at(10)],
             param_dtype=ddp.BF16, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, step_dev=None,
             seed=0, norm=NORM, max_norm=1.0)
    a.update(change)
    return a


def read_args(**change):
    a = dict(numels=[100, 0, 7], m=[at(5, 1), 0, at(6)], v=[at(7), 0, at(8, 3)], scales=[at(11, 2), 0, at(12)],
             m_out=[at(0), 0, at(1)], v_out=[at(2), 0, at(3)], out_dtype=ddp.F32)
    a.update(change)
    return a


ROWS = [
    (dict(P=0), N.DDP_E_ARG, "P = 0"),
    (dict(P=17), N.DDP_E_ARG, "P = 17"),
    (dict(n=-1), N.DDP_E_ARG, "negative"),
    (dict(n=(1 << 40) + 1), N.DDP_E_ARG, "2^40"),
    (dict(rank_codes=None), N.DDP_E_ARG, "rank_codes"),
    (dict(rank_codes=[at(4), 0]), N.DDP_E_ARG, "rank_codes[1]"),
    (dict(rank_codes=[at(4, 8), at(5)]), N.DDP_E_ALIGN, "rank_codes[0]"),
    (dict(rank_scales=None), N.DDP_E_ARG, "rank_scales"),
    (dict(rank_scales=[0, at(7)]), N.DDP_E_ARG, "rank_scales[0]"),
]


@pytest.mark.parametrize("change,status,text", ROWS + [
    (dict(in_dtype=3), N.DDP_E_ARG, "dtype"),
    (dict(residual_dtype=-1), N.DDP_E_ARG, "dtype"),
    (dict(rank_in=None), N.DDP_E_ARG, "rank_in"),
    (dict(rank_in=[at(0), at(1, 2)]), N.DDP_E_ALIGN, "rank_in[1]"),
    (dict(rank_residual=[at(2, 1), at(3)]), N.DDP_E_ALIGN, "rank_residual[0]"),
    (dict(rank_residual=[at(2), 0]), N.DDP_E_ARG, "rank_residual[1]"),
    (dict(rank_codes=[at(4), at(4)]), N.DDP_E_OVERLAP, None),               # both ranks' codes
    (dict(rank_codes=[at(4), at(4, 496)]), N.DDP_E_OVERLAP, None),          # by one 16-byte line
    (dict(rank_codes=[at(0, 3984), at(5)]), N.DDP_E_OVERLAP, None),         # over the gradient's end
    (dict(rank_scales=[at(6), at(6, 31)]), N.DDP_E_OVERLAP, None),
    (dict(rank_residual=[at(0), at(3)]), N.DDP_E_OVERLAP, None),            # the gradient as its residual
    (dict(rank_residual=[at(2), at(2)]), N.DDP_E_OVERLAP, None),            # one residual for two ranks
])
def test_quantize_refusals(change, status, text):
    refused(ddp.mx4_quantize_rows, quantize_args(**change), status, text)


@pytest.mark.parametrize("change,status,text", ROWS + [
    (dict(out_dtype=3), N.DDP_E_ARG, "dtype"),
    (dict(rank_out=None), N.DDP_E_ARG, "rank_out"),
    (dict(rank_out=[at(0, 2), at(1)]), N.DDP_E_ALIGN, "rank_out[0]"),
    (dict(rank_out=[at(0), at(0)]), N.DDP_E_OVERLAP, None),
    (dict(rank_out=[at(0), at(5, 508)]), N.DDP_E_OVERLAP, None),
])
def test_dequantize_refusals(change, status, text):
    refused(ddp.mx4_dequantize_rows, dequantize_args(**change), status, text)


NORMS = [
    (dict(op=2), N.DDP_E_ARG, None),
    (dict(norm=NORM + 2), N.DDP_E_ALIGN, "norm"),
    (dict(workspace=None), N.DDP_E_ARG, "workspace"),
    (dict(workspace_bytes=7), N.DDP_E_ARG, "workspace"),
    (dict(workspace=WS + 8), N.DDP_E_ALIGN, "workspace"),
    (dict(norm=WS + 4), N.DDP_E_OVERLAP, None),
    (dict(norm=at(4, 16)), N.DDP_E_OVERLAP, None),
    (dict(workspace=at(6, 16)), N.DDP_E_OVERLAP, None),
]


@pytest.mark.parametrize("change,status,text", ROWS + [x for x in NORMS if "op" not in x[0]] + [
    (dict(out_dtype=9), N.DDP_E_ARG, "dtype"),
    (dict(P=3, rank_codes=[at(4), at(5), at(12)], rank_scales=[at(6), at(7), at(13)]), N.DDP_E_ARG, "n_out"),
    (dict(rank_out=[at(0), 0]), N.DDP_E_ARG, "rank_out[1]"),
    (dict(rank_out=[at(0), at(1, 2)]), N.DDP_E_ALIGN, "rank_out[1]"),
    (dict(rank_out=[at(0), at(0, 4)]), N.DDP_E_OVERLAP, None),
    (dict(rank_out=[at(4), at(1)]), N.DDP_E_OVERLAP, None),                 # values over codes
])
def test_reduce_refusals(change, status, text):
    refused(ddp.allreduce_mx4_rows, reduce_args(**change), status, text)


def test_unknown_op():
    with pytest.raises(KeyError):
        ddp.allreduce_mx4_rows(**reduce_args(op="max"))
    null = ctypes.cast(None, ctypes.POINTER(ctypes.c_void_p))
    assert N.lib().allreduce_mx4(7, 2, null, null, 0, 1, null, 0, None, None, 0, None) == N.DDP_E_ARG


@pytest.mark.parametrize("change,status,text", ROWS + [x for x in NORMS if "op" not in x[0]] + [
    (dict(residual_dtype=9), N.DDP_E_ARG, "dtype"),
    (dict(residual=at(2, 2)), N.DDP_E_ALIGN, "residual"),
    (dict(residual=at(9)), N.DDP_E_OVERLAP, "residual"),
    (dict(residual=WS), N.DDP_E_OVERLAP, None),
    (dict(out_codes=[at(8), at(9, 4)]), N.DDP_E_ALIGN, "out_codes[1]"),
    (dict(out_codes=[at(8), 0]), N.DDP_E_ARG, "out_codes[1]"),
    (dict(out_scales=[at(10), 0]), N.DDP_E_ARG, "out_scales[1]"),
    (dict(out_codes=[at(4, 16), at(9)]), N.DDP_E_OVERLAP, None),            # inside an input, not on it
    (dict(out_scales=[at(6, 1), at(11)]), N.DDP_E_OVERLAP, None),
    (dict(out_scales=[at(10), at(9)]), N.DDP_E_OVERLAP, None),              # scales over codes
])
def test_coded_reduce_refusals(change, status, text):
    refused(ddp.allreduce_mx4_coded, coded_args(**change), status, text)


def test_coded_reduce_lists():
    with pytest.raises(ValueError):
        ddp.allreduce_mx4_coded(**coded_args(out_scales=[at(10)]))


@pytest.mark.parametrize("change,status,text", [
    (dict(numels=[100, -1, 7]), N.DDP_E_ARG, "negative"),
    (dict(grads=[0, 0, at(2)]), N.DDP_E_ARG, "grads[0]"),
    (dict(grads=[at(0, 1), 0, at(2)]), N.DDP_E_ALIGN, "grads[0]"),
    (dict(w=[at(3, 2), 0, at(4)]), N.DDP_E_ALIGN, "w[0]"),
    (dict(m=[at(5), 0, 0]), N.DDP_E_ARG, "m[2]"),
    (dict(v=[0, 0, at(8)]), N.DDP_E_ARG, "v[0]"),
    (dict(scales=[0, 0, at(12)]), N.DDP_E_ARG, "scales[0]"),
    (dict(scales=[at(11, 1), 0, at(12)]), N.DDP_E_ALIGN, "scales[0]"),
    (dict(m=[at(5), 0, at(5, 99)]), N.DDP_E_OVERLAP, None),
    (dict(v=[at(5, 100), 0, at(8)]), N.DDP_E_OVERLAP, None),                # one byte into m
    (dict(scales=[at(7, 98), 0, at(12)]), N.DDP_E_OVERLAP, None),
    (dict(scales=[at(11), 0, at(11, 6)]), N.DDP_E_OVERLAP, None),           # four blocks are eight bytes
    (dict(params=[at(3), 0, at(10)]), N.DDP_E_OVERLAP, None),
    (dict(grad_dtype=4), N.DDP_E_ARG, "dtype"),
    (dict(param_dtype=4), N.DDP_E_ARG, "dtype"),
    (dict(lr=INF), N.DDP_E_ARG, "lr"),
    (dict(beta1=1.0), N.DDP_E_ARG, "beta1"),
    (dict(beta2=-0.1), N.DDP_E_ARG, "beta2"),
    (dict(eps=NAN), N.DDP_E_ARG, "eps"),
    (dict(step=0), N.DDP_E_ARG, "step"),
    (dict(step_dev=STEPS + 4), N.DDP_E_ALIGN, "step_dev"),
    (dict(step_dev=at(11, 4)), N.DDP_E_ALIGN, None),
    (dict(step_dev=at(5, 8)), N.DDP_E_OVERLAP, None),
    (dict(norm=NORM + 1), N.DDP_E_ALIGN, "norm"),
    (dict(norm=at(12)), N.DDP_E_OVERLAP, None),
    (dict(max_norm=-1.0), N.DDP_E_ARG, "max_norm"),
])
def test_adamw8_refusals(change, status, text):
    refused(ddp.adamw8_step_multi, adamw_args(**change), status, text)


@pytest.mark.parametrize("order", ["lists", "interleaved", "shuffled"])
@pytest.mark.parametrize("pair", [("w", "m"), ("m", "scales"), ("g", "v"), ("w", "w")])
def test_adamw8_overlaps_among_many(order, pair):
    """40 tensors of five lists that lie in order, turn by turn or anywhere:
    one buffer moved a byte (or an element) into another is refused."""
    T, size = 40, {"g": 200, "w": 400, "m": 100, "v": 100, "scales": 8}
    names = list(size)
    slots = [(k, t) for k in names for t in range(T)] if order == "lists" else [(k, t) for t in range(T) for k in names]
    if order == "shuffled":
        import random
        random.Random(1).shuffle(slots)
    place = {slot: BASE + 1024 * i for i, slot in enumerate(slots)}
    one, other = (pair[0], 7), (pair[1], 23)
    place[other] = place[one] + size[pair[0]] - (4 if pair[1] == "w" else 2 if pair[1] in ("g", "scales") else 1)
    lists = {k: [place[k, t] for t in range(T)] for k in names}
    refused(ddp.adamw8_step_multi, adamw_args(numels=[100] * T, grads=lists["g"], w=lists["w"], m=lists["m"], v=lists["v"],
                                              scales=lists["scales"], params=None, norm=None), N.DDP_E_OVERLAP)


def test_adamw8_null_lists():
    assert N.lib().adamw8_step_multi(1, (ctypes.c_int64 * 1)(5), N.pointer_array([at(0)]), 0, N.pointer_array([at(1)]),
                                     N.pointer_array([at(2)]), N.pointer_array([at(3)]), None, None, 0, 1e-3, 0.9, 0.9,
                                     1e-8, 0.0, 1, None, 0, None, 0.0, None) == N.DDP_E_ARG
    with pytest.raises(ValueError):
        ddp.adamw8_step_multi(**adamw_args(scales=[at(11)]))
    with pytest.raises(ValueError):
        ddp.adamw8_read_multi(**read_args(v_out=[at(2)]))


@pytest.mark.parametrize("change,status,text", [
    (dict(numels=[100, 1 << 41, 7]), N.DDP_E_ARG, "2^40"),
    (dict(out_dtype=2), N.DDP_E_ARG, "dtype"),
    (dict(m=[0, 0, at(6)]), N.DDP_E_ARG, "m[0]"),
    (dict(scales=[at(11, 1), 0, at(12)]), N.DDP_E_ALIGN, "scales[0]"),
    (dict(m_out=[at(0, 2), 0, at(1)]), N.DDP_E_ALIGN, "m_out[0]"),
    (dict(v_out=[at(0, 396), 0, at(3)]), N.DDP_E_OVERLAP, None),
    (dict(v_out=[at(7), 0, at(3)]), N.DDP_E_OVERLAP, None),
    (dict(m_out=[at(11), 0, at(1)]), N.DDP_E_OVERLAP, None),
])
def test_read_refusals(change, status, text):
    refused(ddp.adamw8_read_multi, read_args(**change), status, text)


def test_workspace():
    assert ddp.allreduce_mx4_workspace_bytes(0) == 0
    assert ddp.allreduce_mx4_workspace_bytes(1) == 8
    assert ddp.allreduce_mx4_workspace_bytes(2049) == 16
    assert ddp.allreduce_mx4_workspace_bytes(1 << 40) <= 1 << 27
    for n in (-1, (1 << 40) + 1):
        with pytest.raises(DdpError):
            ddp.allreduce_mx4_workspace_bytes(n)
    assert N.lib().allreduce_mx4_workspace_bytes(5, None) == N.DDP_E_ARG


def test_nothing_to_do_without_buffers():
    null = ctypes.cast(None, ctypes.POINTER(ctypes.c_void_p))
    lib = N.lib()
    assert lib.mx4_quantize(2, null, 0, 0, null, 0, null, null, None) == N.DDP_OK
    assert lib.mx4_dequantize(2, null, null, 0, null, 0, None) == N.DDP_OK
    assert lib.allreduce_mx4(1, 2, null, null, 0, 2, null, 0, None, None, 0, None) == N.DDP_OK
    assert lib.allreduce_mx4_coded(1, 2, null, null, 0, 1, null, null, None, 0, None, None, 0, None) == N.DDP_OK


# ----------------------------------------------------- tensor level ----

class Gpu(torch.Tensor):
    """A CPU tensor that says it lives on the GPU."""
    is_cuda = True


def gpu(n, dtype=torch.uint8):
    return torch.Tensor._make_subclass(Gpu, torch.zeros(n, dtype=dtype))


def test_mx4_sizes():
    x = ddp.Mx4(gpu(64), gpu(4), 100)
    assert x.numel == 100
    y = x.narrow(32, 68)
    assert y.numel == 68 and y.codes.numel() == 48 and y.scales.numel() == 3
    assert x.narrow(64, 0).numel == 0 and x.narrow(96, 4).codes.numel() == 16
    for bad in ((1, 32), (32, 33), (0, 101), (-32, 64), (64, -32)):
        with pytest.raises(ValueError):
            x.narrow(*bad)
    for codes, scales, n in ((gpu(63), gpu(4), 100), (gpu(64), gpu(3), 100), (gpu(64), gpu(4), 129),
                             (torch.zeros(64, dtype=torch.uint8), gpu(4), 100), (gpu(128)[::2], gpu(4), 100)):
        with pytest.raises(ValueError):
            ddp.Mx4(codes, scales, n)
    with pytest.raises(TypeError):
        ddp.Mx4(gpu(64, torch.int8), gpu(4), 100)
    with pytest.raises(ValueError):
        ddp.Mx4.empty(-1, "cpu")
    with pytest.raises(ValueError, match="negative"):
        ddp.Mx4(gpu(0), gpu(0), -1)


@pytest.mark.parametrize("fn, args, short", [
    (ddp.mx4_quantize_rows, quantize_args, ("rank_in", "rank_residual", "rank_codes", "rank_scales")),
    (ddp.mx4_dequantize_rows, dequantize_args, ("rank_codes", "rank_scales", "rank_out")),
    (ddp.allreduce_mx4_rows, reduce_args, ("rank_codes", "rank_scales")),
    (ddp.allreduce_mx4_coded, coded_args, ("rank_codes", "rank_scales"))])
def test_fewer_addresses_than_ranks_are_refused(fn, args, short):
    for name in short:
        with pytest.raises(ValueError, match="need 2 addresses, got 1"):
            fn(**args(**{name: [at(20)]}))


def test_moments8_sizes():
    ddp.Moments8([gpu(100), gpu(0)], [gpu(100), gpu(0)], [gpu(8), gpu(0)])
    for m, v, s in (([gpu(100)], [gpu(99)], [gpu(8)]), ([gpu(100)], [gpu(100)], [gpu(4)]),
                    ([gpu(100)], [gpu(100)] * 2, [gpu(8)]), ([], [], [])):
        with pytest.raises(ValueError):
            ddp.Moments8(m, v, s)
    with pytest.raises(TypeError):
        ddp.Moments8([gpu(100, torch.float32)], [gpu(100)], [gpu(8)])
    with pytest.raises(ValueError):
        ddp.Moments8.zeros([])


def test_tensor_level_refusals(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # a CPU tensor's
    row = ddp.Mx4(gpu(64), gpu(4), 100)
    with pytest.raises(TypeError):
        ddp.mx4_dequantize([gpu(64)])
    with pytest.raises(ValueError):
        ddp.mx4_dequantize([])
    with pytest.raises(ValueError):
        ddp.mx4_dequantize([row, ddp.Mx4(gpu(16), gpu(1), 20)])
    with pytest.raises(ValueError):
        ddp.allreduce_mx4([row] * 17)
    with pytest.raises(ValueError):
        ddp.mx4_quantize([gpu(100, torch.float32)], out=[row, row])
    mom = ddp.Moments8([gpu(100)], [gpu(100)], [gpu(8)])
    mg = ddp.MultiGrad(gpu(100, torch.float32))
    w = gpu(100, torch.float32)
    with pytest.raises(TypeError):
        mg.bind_adamw8(w, (gpu(100), gpu(100), gpu(8)))
    with pytest.raises(ValueError):
        ddp.MultiGrad(gpu(99, torch.float32)).bind_adamw8(gpu(99, torch.float32), mom)
    with pytest.raises(TypeError):
        mg.bind_adamw(w, None, w)
    with pytest.raises(TypeError):
        mg.bind_adamw(w, w, None)
    run = mg.bind_adamw8(w, mom)
    with pytest.raises(ValueError):
        run(1e-3, 1, max_norm=1.0)
    w.data = torch.zeros(100)
    with pytest.raises(ValueError, match="bind it again"):
        run(1e-3, 1)


def test_resized_storages_are_refused():
    codes, scales = gpu(64), gpu(4)
    row = ddp.Mx4(codes, scales, 100)
    part = row.narrow(32, 32)
    scales.untyped_storage().resize_(0)
    for r in (row, part):
        with pytest.raises(ValueError, match="resized"):
            ddp.mx4_dequantize([r])
    m = gpu(100)
    mom = ddp.Moments8([m], [gpu(100)], [gpu(8)])
    run = ddp.MultiGrad(gpu(100, torch.float32)).bind_adamw8(gpu(100, torch.float32), mom)
    m.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="resized"):
        run(1e-3, 1)


def test_objects_keep_the_memory_they_were_made_of():
    """A tensor that is given other memory, or another size in the same, is no
    longer a part of the object; the object's own views are."""
    codes, m = gpu(64), gpu(100)
    row, mom = ddp.Mx4(codes, gpu(4), 100), ddp.Moments8([m], [gpu(100)], [gpu(8)])
    at, mom_at = row.codes_at, list(mom._held[0].at)
    assert at == codes.data_ptr() == row.codes.data_ptr() and mom_at == [m.data_ptr()] == [mom.m[0].data_ptr()]
    codes.data = torch.zeros(64, dtype=torch.uint8)
    m.resize_(50)
    mom.m[0].data = torch.zeros(100, dtype=torch.uint8)
    assert row.codes_at == at == row.codes.data_ptr() and row.codes.numel() == 64
    assert mom.m[0].data_ptr() == mom_at[0] and mom.m[0].numel() == 100
    rows = ddp.Mx4.rows(3, 1000, "cpu")
    assert all(r.codes.numel() == 512 and r.scales.numel() == 32 and r.codes_at % 16 == rows[0].codes_at % 16 for r in rows)
    assert len({r.codes_at for r in rows} | {r.scales_at for r in rows}) == 6


# ---------------------------------------------- what the calls hold ----

class Lib:
    """The library with its launching calls written down instead of made."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("adamw_step_multi", "adamw8_step_multi", "adamw8_read_multi", "mx4_quantize", "mx4_dequantize",
                    "allreduce_mx4", "allreduce_mx4_coded"):
            return lambda *args: self.calls.append((name, args)) or N.DDP_OK
        return getattr(self.real, name)


@pytest.fixture
def lib(monkeypatch):
    from gradient_all_reduce_allreduce_amd import api
    stub = Lib(N.lib())
    monkeypatch.setattr(N, "lib", lambda: stub)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)    # a CPU tensor's device index
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    return stub


def step8(g, params=None):
    f32 = [gpu(x.numel(), torch.float32) for x in g]
    mom = ddp.Moments8([gpu(x.numel()) for x in g], [gpu(x.numel()) for x in g], [gpu(2 * -(-x.numel() // 32)) for x in g])
    return f32, mom


def test_eight_bit_state_never_goes_to_the_32_bit_step(lib):
    """Whatever is given for the seed: 8-bit moments reach their own call, or
    the call is refused."""
    g = [gpu(100, torch.float32), gpu(7, torch.float32)]
    w, mom = step8(g)
    run = ddp.MultiGrad(g).bind_adamw8(w, mom)
    run(1e-3, 1)
    run(1e-3, 1, seed=-5)
    run(1e-3, 1, seed=True)
    for bad in (None, 1.5, "1"):
        with pytest.raises(TypeError):
            run(1e-3, 1, seed=bad)
    assert [name for name, _ in lib.calls] == ["adamw8_step_multi"] * 3
    assert [args[17] for _, args in lib.calls] == [0, -5, 1]
    args = lib.calls[0][1]
    assert list(args[5]) == [x.data_ptr() for x in mom.m] and list(args[7]) == [x.data_ptr() for x in mom.scales]


def test_nothing_outlives_a_step(lib):
    import gc
    import weakref
    gc.disable()
    try:
        for bound in (False, True):
            g = [gpu(100, torch.float32)]
            w, mom = step8(g)
            refs = [weakref.ref(x) for x in (*g, *w, mom)]
            if bound:
                run = ddp.MultiGrad(g).bind_adamw8(w, mom)
                run(1e-3, 1)
                read = mom.bind_read(gpu(100, torch.float32), gpu(100, torch.float32))
                read()
                del run, read
            else:
                ddp.adamw8_step(g, w, mom, 1e-3, 1)
            del g, w, mom
            assert all(r() is None for r in refs), bound
    finally:
        gc.enable()


def test_a_bound_step_keeps_its_memory(lib):
    import weakref
    g = [gpu(100, torch.float32)]
    w, mom = step8(g)
    storages = [x.data_ptr() for x in (mom.m[0], w[0])]
    run = ddp.MultiGrad(g).bind_adamw8(w, mom)
    held = weakref.ref(g[0])
    del g, w, mom
    assert held() is not None
    run(1e-3, 2)
    assert [lib.calls[-1][1][5][0], lib.calls[-1][1][4][0]] == storages


# ------------------------------- lists that lie in any order in memory ----

SIZES8 = {"grads": 200, "w": 400, "m": 100, "v": 100, "scales": 8, "params": 200}      # bytes of 100 elements


def lists_at(order, T):
    """Addresses of T tensors in each of the six lists, every list whole and in
    order, the lists in the given order in memory."""
    return {k: [BASE + (order.index(k) * T + t) * 1024 for t in range(T)] for k in SIZES8}


def step8_of(lists, T):
    """The call on such lists, without what Python does for it."""
    arrays = {k: N.pointer_array(x) for k, x in lists.items()}
    numels, call = (ctypes.c_int64 * T)(*[100] * T), N.lib().adamw8_step_multi
    args = (T, numels, arrays["grads"], ddp.BF16, arrays["w"], arrays["m"], arrays["v"], arrays["scales"],
            arrays["params"], ddp.BF16, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, None, 0, None, 0.0, None)
    return lambda: call(*args)


@pytest.mark.parametrize("which", range(24))
def test_adamw8_overlaps_in_any_order_of_lists(which):
    """Lists in any order in memory: one buffer moved a byte (or an element)
    into its own list's or another list's is refused, before any launch."""
    import itertools
    order = list(itertools.permutations(SIZES8))[which * 29 + 1]
    T = 9
    for one, other in itertools.product(SIZES8, repeat=2):
        for t, u in ((0, T - 1), (T - 1, 0), (4, 5)):
            if one == other == "grads":
                continue            # read only
            lists = lists_at(order, T)
            lists[other][u] = lists[one][t] + SIZES8[one] - {"w": 4, "m": 1, "v": 1}.get(other, 2)
            refused(ddp.adamw8_step_multi, adamw_args(numels=[100] * T, norm=None, **lists), N.DDP_E_OVERLAP, "overlaps")


def test_whole_lists_need_no_sorting_in_any_order():
    """What the overlap check takes where every list lies whole and in order,
    whatever the lists' order among each other, is near what it takes where one
    lies behind the other (sorted they took up to 5 times as long).  The last copy
    overlaps the one before it, so that no call gets past the check."""
    import random
    import time

    def host_time(order, T=1200):
        lists = lists_at(order, T)
        lists["params"][-1] = lists["params"][-2] + 198
        call = step8_of(lists, T)
        best = 1e9
        for _ in range(40):
            start = time.perf_counter()
            status = call()
            best = min(best, time.perf_counter() - start)
            assert status == N.DDP_E_OVERLAP
        return best

    names = list(SIZES8)
    in_order = host_time(names)
    orders = [random.Random(k).sample(names, 6) for k in range(8)] + [names[::-1], ["params", "grads", "m", "v", "scales", "w"]]
    for order in orders:
        assert host_time(order) < 2.5 * in_order, order


def test_one_output_without_a_list(lib):
    """A single copy may be given as the tensor or the Mx4 itself; a tensor of
    rows is still a list of them."""
    class OnDevice(Gpu):
        def get_device(self):
            return None                                 # as its device's index

    def f32(*shape):
        return torch.Tensor._make_subclass(OnDevice, torch.zeros(*shape))

    rows = [ddp.Mx4(gpu(64), gpu(4), 100) for _ in range(3)]
    grad, coded = f32(100), ddp.Mx4(gpu(64), gpu(4), 100)
    assert ddp.allreduce_mx4(rows, "mean", out=grad)[0] is grad
    assert ddp.allreduce_mx4(rows, "mean", out=[grad])[0] is grad
    assert ddp.allreduce_mx4(rows, "mean", out=coded, residual=f32(100))[0] is coded
    (name, args), again, (coded_name, coded_args) = lib.calls
    assert name == "allreduce_mx4" and (args[5], args[6][0]) == (1, grad.data_ptr())
    assert again[1][5] == 1 and again[1][6][0] == grad.data_ptr()
    assert coded_name == "allreduce_mx4_coded" and (coded_args[5], coded_args[6][0]) == (1, coded.codes_at)
    assert len(ddp.allreduce_mx4(rows, "sum", out=f32(3, 100))) == 3 and lib.calls[-1][1][5] == 3
    for wrong in (f32(99), f32(101)):
        with pytest.raises(ValueError, match="out must match"):
            ddp.allreduce_mx4(rows, out=wrong)
    ones = [ddp.Mx4(gpu(16), gpu(1), 1) for _ in range(3)]
    assert len(ddp.allreduce_mx4(ones, out=f32(3))) == 3 and len(ddp.allreduce_mx4(ones, out=f32(1))) == 1
