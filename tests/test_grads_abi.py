"""Refusals of the gradient norm, clipping, all-reduce with norm and AdamW
calls: host only, every call returns before any launch."""

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


def norm_args(**change):
    a = dict(numels=[200_000, 0, 7], ptrs=[at(0), 0, at(2)], dtypes=[ddp.F32, ddp.BF16, ddp.BF16], workspace=WS,
             workspace_bytes=ddp.NORM_WORKSPACE_BYTES, norm=NORM)
    a.update(change)
    return a


def clip_args(**change):
    a = norm_args(out=[at(4), 0, at(6)], max_norm=1.0, norm_given=False)
    a.update(change)
    return a


def adamw_args(**change):
    a = dict(numels=[100, 0, 7], grads=[at(0), 0, at(2)], grad_dtype=ddp.BF16, w=[at(3), 0, at(4)],
             m=[at(5), 0, at(6)], v=[at(7), 0, at(8)], params=[at(9), 0, at(10)], param_dtype=ddp.BF16, lr=1e-3,
             beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, step_dev=None, norm=NORM, max_norm=1.0)
    a.update(change)
    return a


def ring_args(**change):
    a = dict(op="mean", P=2, chunking=2, rank_in=[at(0), at(1)], in_dtype=ddp.F32, rank_out=[at(2), at(3)],
             out_dtype=ddp.F32, n=1000, norm=NORM, workspace=WS, workspace_bytes=1 << 20)
    a.update(change)
    return a


def refused(fn, args, status, text=None):
    with pytest.raises(DdpError) as e:
        fn(**args)
    assert e.value.status == status, e.value
    if text:
        assert text in str(e.value)


LISTS = [
    (dict(numels=[200_000, -1, 7]), N.DDP_E_ARG, "negative"),
    (dict(numels=[(1 << 40) + 1, 0, 7]), N.DDP_E_ARG, "2^40"),
    (dict(numels=[], ptrs=[], dtypes=[]), N.DDP_E_ARG, "n_tensors"),
    (dict(ptrs=[0, 0, at(2)]), N.DDP_E_ARG, "NULL"),
    (dict(ptrs=[at(0, 2), 0, at(2)]), N.DDP_E_ALIGN, "ptrs[0]"),
    (dict(ptrs=[at(0), 0, at(2, 1)]), N.DDP_E_ALIGN, "ptrs[2]"),
    (dict(dtypes=[ddp.F32, 5, ddp.BF16]), N.DDP_E_ARG, "dtypes[1]"),
    (dict(norm=None), N.DDP_E_ARG, "norm"),
    (dict(norm=NORM + 2), N.DDP_E_ALIGN, "norm"),
    (dict(norm=at(0, 396)), N.DDP_E_OVERLAP, None),
    (dict(workspace=None), N.DDP_E_ARG, "workspace"),
    (dict(workspace=WS + 8), N.DDP_E_ALIGN, "workspace"),
    (dict(workspace_bytes=ddp.NORM_WORKSPACE_BYTES - 1), N.DDP_E_ARG, "workspace"),
    (dict(workspace=at(0, 384)), N.DDP_E_OVERLAP, None),
    (dict(norm=WS + 16), N.DDP_E_OVERLAP, None),
]


@pytest.mark.parametrize("change,status,text", LISTS)
def test_norm_refusals(change, status, text):
    refused(ddp.grad_norm_multi, norm_args(**change), status, text)


@pytest.mark.parametrize("change,status,text", [x for x in LISTS if "numels" not in x[0] or x[0]["numels"]] + [
    (dict(max_norm=-1.0), N.DDP_E_ARG, "max_norm"),
    (dict(max_norm=NAN), N.DDP_E_ARG, "max_norm"),
    (dict(out=[at(4), 0, 0]), N.DDP_E_ARG, "out[2]"),
    (dict(out=[at(4, 2), 0, at(6)]), N.DDP_E_ALIGN, "out[0]"),
    (dict(out=[at(0, 4), 0, at(6)]), N.DDP_E_OVERLAP, None),        # over its own input, not in place
    (dict(out=[at(2), 0, at(6)]), N.DDP_E_OVERLAP, None),           # another tensor's input
    (dict(out=[at(4), 0, at(4, 799_998)]), N.DDP_E_OVERLAP, None),      # two outputs, by one element
    # the same tensor twice, in place
    (dict(numels=[9, 9, 0], ptrs=[at(0), at(0), 0], dtypes=[ddp.F32] * 3, out=[at(0), at(0), 0]),
     N.DDP_E_OVERLAP, None),
    (dict(norm_given=True, norm=None), N.DDP_E_ARG, "norm"),
    (dict(norm_given=True, norm=at(4)), N.DDP_E_OVERLAP, None),     # an output over the given norm
])
def test_clip_refusals(change, status, text):
    refused(ddp.grad_clip_multi, clip_args(**change), status, text)


@pytest.mark.parametrize("change,status,text", [
    (dict(numels=[100, -1, 7]), N.DDP_E_ARG, "negative"),
    (dict(grads=[0, 0, at(2)]), N.DDP_E_ARG, "grads[0]"),
    (dict(grads=[at(0, 1), 0, at(2)]), N.DDP_E_ALIGN, "grads[0]"),
    (dict(w=[at(3, 2), 0, at(4)]), N.DDP_E_ALIGN, "w[0]"),
    (dict(m=[at(5), 0, 0]), N.DDP_E_ARG, "m[2]"),
    (dict(v=[at(7), 0, at(8, 2)]), N.DDP_E_ALIGN, "v[2]"),
    (dict(params=[at(9, 1), 0, at(10)]), N.DDP_E_ALIGN, "params[0]"),
    (dict(grad_dtype=7), N.DDP_E_ARG, "dtype"),
    (dict(param_dtype=-1), N.DDP_E_ARG, "dtype"),
    (dict(w=[at(5), 0, at(4)]), N.DDP_E_OVERLAP, None),             # w[0] is m[0]
    (dict(v=[at(7), 0, at(7, 396)]), N.DDP_E_OVERLAP, None),
    (dict(params=[at(0), 0, at(10)]), N.DDP_E_OVERLAP, None),       # over its gradient
    (dict(norm=at(5)), N.DDP_E_OVERLAP, None),
    (dict(step_dev=at(7)), N.DDP_E_OVERLAP, None),
    (dict(step_dev=STEPS + 4), N.DDP_E_ALIGN, "step_dev"),
    (dict(step=0), N.DDP_E_ARG, "step"),
    (dict(lr=INF), N.DDP_E_ARG, "lr"),
    (dict(weight_decay=NAN), N.DDP_E_ARG, "weight_decay"),
    (dict(beta1=1.0), N.DDP_E_ARG, "beta1"),
    (dict(beta2=-0.1), N.DDP_E_ARG, "beta2"),
    (dict(beta2=NAN), N.DDP_E_ARG, "beta2"),
    (dict(eps=-1e-8), N.DDP_E_ARG, "eps"),
    (dict(eps=INF), N.DDP_E_ARG, "eps"),
    (dict(max_norm=-1.0), N.DDP_E_ARG, "max_norm"),
    (dict(norm=NORM + 1), N.DDP_E_ALIGN, "norm"),
])
def test_adamw_refusals(change, status, text):
    refused(ddp.adamw_step_multi, adamw_args(**change), status, text)


@pytest.mark.parametrize("change,status,text", [
    (dict(P=0, rank_in=[], rank_out=[]), N.DDP_E_ARG, "P = 0"),
    (dict(chunking=0), N.DDP_E_ARG, "chunking"),
    (dict(n=-1), N.DDP_E_ARG, "negative"),
    (dict(in_dtype=9), N.DDP_E_ARG, "dtype"),
    (dict(rank_in=[at(0), at(1, 4)]), N.DDP_E_ALIGN, "rank_in[1]"),
    (dict(rank_out=[at(2), 0]), N.DDP_E_ARG, "rank_out[1]"),
    (dict(rank_out=[at(2), at(3), at(4)]), N.DDP_E_ARG, "n_out"),
    (dict(rank_out=[at(0, 16)]), N.DDP_E_OVERLAP, None),
    (dict(norm=None), N.DDP_E_ARG, "norm"),
    (dict(norm=at(2, 400)), N.DDP_E_OVERLAP, "norm"),
    (dict(workspace=None), N.DDP_E_ARG, "workspace"),
    (dict(workspace=at(1)), N.DDP_E_OVERLAP, "workspace"),
    (dict(workspace=NORM - 16), N.DDP_E_OVERLAP, "workspace"),
    (dict(workspace_bytes=8), N.DDP_E_ARG, "workspace"),
])
def test_allreduce_norm_refusals(change, status, text):
    refused(ddp.allreduce_ring_norm, ring_args(**change), status, text)
    refused(ddp.allreduce_ring_norm_buckets, ring_args(bucket_elems=256, **change), status, text)


def test_bucket_size_refusals():
    refused(ddp.allreduce_ring_norm_buckets, ring_args(bucket_elems=0), N.DDP_E_ARG, "bucket_elems")
    refused(ddp.allreduce_ring_norm_buckets, ring_args(bucket_elems=3), N.DDP_E_ALIGN, "bucket_elems")


def test_workspace_bytes_grow_with_the_workgroups():
    f = ddp.allreduce_norm_workspace_bytes
    assert f(8, 8, ddp.F32, ddp.F32, 0) == 0
    assert f(8, 8, ddp.F32, ddp.F32, 1) == 8
    # 256-element tiles at P = 8; 64 elements per workgroup where the ring's
    # chunks are shorter than a tile
    assert f(8, 8, ddp.F32, ddp.F32, 256 * 1000) == 8000
    assert f(8, 8, ddp.F32, ddp.F32, 640) == 80
    # past 4,096 workgroups the sum has a second level: 64 sums and a count
    assert f(8, 8, ddp.F32, ddp.F32, 256 * 20000) == 8 * (20000 + 65)
    # buckets that are one ring need no more than the flat buffer
    assert f(8, 8, ddp.F32, ddp.F32, 4 * 8192, 8192) == f(8, 8, ddp.F32, ddp.F32, 4 * 8192)
    with pytest.raises(DdpError):
        f(8, 0, ddp.F32, ddp.F32, 10)
    with pytest.raises(DdpError):
        f(8, 8, ddp.F32, ddp.F32, 10, 3)


def test_norm_workspace_bytes():
    f = ddp.grad_norm_workspace_bytes
    tile = 4096
    assert f([64 * tile // 4], [at(0)], [ddp.F32]) == 0 and f([64 * tile // 2], [at(0)], [ddp.BF16]) == 0
    assert f([64 * tile // 4 + 1], [at(0)], [ddp.F32]) == ddp.NORM_WORKSPACE_BYTES
    # off a line by one element: one piece more
    assert f([64 * tile // 4], [at(0, 4)], [ddp.F32]) == ddp.NORM_WORKSPACE_BYTES
    assert f([64 * tile // 4 - 1], [at(0, 4)], [ddp.F32]) == 0
    assert f([1] * 64 + [0], [at(k) for k in range(65)], [ddp.F32] * 65) == 0
    assert f([1] * 65, [at(k) for k in range(65)], [ddp.F32] * 65) == ddp.NORM_WORKSPACE_BYTES
    with pytest.raises(DdpError):
        f([-1], [at(0)], [ddp.F32])
    with pytest.raises(DdpError):
        f([1], [at(0)], [3])


def test_python_refusals():
    cpu = torch.zeros(4)
    for call in (lambda: ddp.grad_norm([]), lambda: ddp.grad_norm([cpu]), lambda: ddp.grad_norm(cpu),
                 lambda: ddp.clip_grads([cpu], 1.0), lambda: ddp.adamw_step([cpu], [cpu], [cpu], [cpu], 1e-3, 1),
                 lambda: ddp.allreduce_norm([cpu, cpu]), lambda: ddp.allreduce_norm([])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        ddp.grad_norm_multi([1, 2], [at(0)], [0, 0], WS, 1 << 14, NORM)
    with pytest.raises(ValueError):
        ddp.adamw_step_multi(**adamw_args(params=[at(9)]))


def test_nothing_launched_without_gpu():
    """Validation comes first: the calls above made no HIP call, and a list
    past any memory is a status, not an exception through the C boundary."""
    lib = N.lib()
    one = (ctypes.c_int64 * 1)(5)
    assert lib.grad_norm_multi(0, one, None, None, None, 0, None, None) == N.DDP_E_ARG
    assert lib.grad_norm_multi(1, None, None, None, None, 0, None, None) == N.DDP_E_ARG
    assert lib.grad_norm_multi(1, one, None, None, None, 0, None, None) == N.DDP_E_ARG
    assert lib.grad_clip_multi(1, one, None, None, None, 1.0, 0, None, None, 0, None) == N.DDP_E_ARG
    assert lib.adamw_step_multi(1, one, None, 0, None, None, None, None, 0, 1e-3, 0.9, 0.9, 1e-8, 0.0, 1, None,
                                None, 0.0, None) == N.DDP_E_ARG
