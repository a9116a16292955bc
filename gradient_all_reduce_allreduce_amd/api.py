"""Python binding of the C ABI: the same entry points, argument marshalling
only.  Every step of the all-reduce runs in the HIP library; PyTorch is used
here for device memory, pointers and the current stream.

Raw entry points (same names and argument order as the C header, pointers as
Python ints, stream as an int handle or None):
    ddp_bucket_plan, ddp_bucket_pack, ddp_bucket_unpack,
    allreduce_ring_emulated, allreduce_fused_sgd, allreduce_ring_buckets,
    allreduce_fused_sgd_buckets, zero1_sgd_step_emulated, zero1_sgd_step_buckets,
    ddp_buckets_launch_count,
    reducescatter_ring_emulated, reducescatter_ring_buckets,
    allgather_ring_emulated, allgather_ring_buckets, allreduce_ring_stepwise,
    allreduce_ring_stepwise_buckets, allreduce_tree_emulated, allreduce_hierarchical_buckets,
    allreduce_hierarchical_emulated, ddp_multi_plan, ddp_multi_block_map, allreduce_multi_ring_emulated,
    allreduce_multi_fused_sgd, allreduce_multi_ring_noalloc, grad_norm_multi, grad_clip_multi,
    allreduce_ring_norm, allreduce_ring_norm_buckets, allreduce_norm_workspace_bytes,
    adamw_step_multi, grad_norm_workspace_bytes, mx4_quantize_rows, mx4_dequantize_rows,
    allreduce_mx4_rows, allreduce_mx4_coded, allreduce_mx4_workspace_bytes, adamw8_step_multi,
    adamw8_read_multi, ddp_set_wg_per_cu
(mx4_quantize, mx4_dequantize and allreduce_mx4 of the C header end in _rows here: the tensor-level helpers have the
short names.)
Tensor-level helpers:
    allreduce(tensors, op, chunking, out)            -> list of outputs
    allreduce_sgd(grads, w, v, lr, mu, op, chunking, out)
    zero1_sgd_step(grads, w, v, lr, mu, params, op, chunking)
    reduce_scatter, all_gather, allreduce_stepwise, allreduce_tree,
    allreduce_hierarchical, MultiAllReduce
    allreduce_norm(tensors, op, chunking, out)       -> (outputs, norm)
    grad_norm(grads), clip_grads(grads, max_norm), adamw_step(grads, w, m, v, lr, step),
    MultiGrad(grads)
    mx4_quantize(tensors, residual), mx4_dequantize(coded), allreduce_mx4(coded, op, out),
    allreduce_mx4_norm(coded, op, out)               -> (outputs, norm); see mx4.py
    adamw8_step(grads, w, moments, lr, step), Moments8
"""

import ctypes
import functools
import operator

import numpy as np

from . import _native as N

SUM = N.DDP_SUM
MEAN = N.DDP_MEAN
F32 = N.DDP_F32
BF16 = N.DDP_BF16
MAX_RANKS = N.DDP_MAX_RANKS
NORM_WORKSPACE_BYTES = N.DDP_NORM_WORKSPACE_BYTES
MX_BLOCK = N.DDP_MX_BLOCK


class DdpError(RuntimeError):
    """A non-OK status from the library; ``status`` holds the code."""

    def __init__(self, status, message):
        super().__init__(f"{N.STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(status):
    if status != N.DDP_OK:
        raise DdpError(status, N.last_error())


def _op(op):
    if op in (SUM, MEAN):
        return op
    return {"sum": SUM, "mean": MEAN}[op]


# ----------------------------------------------------------- raw entry ----

SEGMENT_DTYPE = np.dtype([("tensor", "<i4"), ("bucket", "<i4"), ("src_off", "<i8"),
                          ("dst_off", "<i8"), ("len", "<i8")])
assert SEGMENT_DTYPE.itemsize == ctypes.sizeof(N.Segment)


def ddp_bucket_plan(numels, dtype, bucket_bytes):
    """Plan buckets (host only).  Returns (segments, n_buckets, total_elems,
    fingerprint); segments is a numpy structured array in the C layout."""
    numels = np.ascontiguousarray(numels, dtype=np.int64)
    T = int(numels.size)
    c_numels = numels.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))
    n_segs = ctypes.c_int64(0)
    n_buckets = ctypes.c_int32(0)
    total = ctypes.c_int64(0)
    fp = ctypes.c_uint64(0)
    lib = N.lib()
    _check(lib.ddp_bucket_plan(c_numels, T, dtype, bucket_bytes, None, 0, ctypes.byref(n_segs),
                               ctypes.byref(n_buckets), ctypes.byref(total), ctypes.byref(fp)))
    segs = np.zeros(n_segs.value, dtype=SEGMENT_DTYPE)
    _check(lib.ddp_bucket_plan(c_numels, T, dtype, bucket_bytes,
                               segs.ctypes.data_as(ctypes.POINTER(N.Segment)), segs.size,
                               ctypes.byref(n_segs), ctypes.byref(n_buckets),
                               ctypes.byref(total), ctypes.byref(fp)))
    return segs, n_buckets.value, total.value, fp.value


def _host_addr(x, dtype=None):
    """Address of a host array: a numpy array (converted to ``dtype`` if
    given), a ctypes object or an int address; None stays NULL."""
    if x is None or isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        if dtype is not None and x.dtype != dtype:
            raise TypeError(f"expected a {dtype} array, got {x.dtype}")
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("host arrays must be contiguous")
        return x.ctypes.data
    return ctypes.addressof(x)


def _ptr_array(ptrs):
    if isinstance(ptrs, ctypes.Array):
        return ptrs
    return N.pointer_array(ptrs)


def ddp_bucket_pack(P, dtype, segs, n_segs, numels, n_tensors, tensor_ptrs, rank_bucket, bucket_len,
                    stream=None):
    """segs: the bucket's segments (a SEGMENT_DTYPE numpy array or a host
    address); numels: int64 numpy array (or address); tensor_ptrs: P *
    n_tensors device addresses, rank-major (a list or a ctypes array)."""
    _check(N.lib().ddp_bucket_pack(P, dtype, _host_addr(segs, SEGMENT_DTYPE), n_segs,
                                   _host_addr(numels, np.int64), n_tensors, _ptr_array(tensor_ptrs),
                                   N.pointer_array(rank_bucket), bucket_len, stream))


def ddp_bucket_unpack(P, dtype, segs, n_segs, numels, n_tensors, tensor_ptrs, rank_bucket, bucket_len,
                      stream=None):
    _check(N.lib().ddp_bucket_unpack(P, dtype, _host_addr(segs, SEGMENT_DTYPE), n_segs,
                                     _host_addr(numels, np.int64), n_tensors, _ptr_array(tensor_ptrs),
                                     N.pointer_array(rank_bucket), bucket_len, stream))


def allreduce_ring_emulated(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n,
                            stream=None):
    _check(N.lib().allreduce_ring_emulated(_op(op), P, chunking, N.pointer_array(rank_in),
                                           in_dtype, N.pointer_array(rank_out), out_dtype, n,
                                           stream))


def allreduce_fused_sgd(op, P, chunking, rank_grad, grad_dtype, n, master_w, momentum, lr, mu,
                        rank_grad_out, out_dtype, stream=None):
    out = N.pointer_array(rank_grad_out) if rank_grad_out is not None else None
    _check(N.lib().allreduce_fused_sgd(_op(op), P, chunking, N.pointer_array(rank_grad),
                                       grad_dtype, n, master_w, momentum, lr, mu, out,
                                       out_dtype, stream))


def allreduce_ring_buckets(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n, bucket_elems,
                           stream=None):
    _check(N.lib().allreduce_ring_buckets(_op(op), P, chunking, N.pointer_array(rank_in), in_dtype,
                                          N.pointer_array(rank_out), out_dtype, n, bucket_elems, stream))


def allreduce_fused_sgd_buckets(op, P, chunking, rank_grad, grad_dtype, n, bucket_elems, master_w,
                                momentum, lr, mu, rank_grad_out, out_dtype, stream=None):
    out = N.pointer_array(rank_grad_out) if rank_grad_out is not None else None
    _check(N.lib().allreduce_fused_sgd_buckets(_op(op), P, chunking, N.pointer_array(rank_grad),
                                               grad_dtype, n, bucket_elems, master_w, momentum, lr, mu,
                                               out, out_dtype, stream))


def zero1_sgd_step_emulated(op, P, chunking, rank_grad, grad_dtype, n, master_w, momentum, lr, mu,
                            rank_param_out, param_dtype, stream=None):
    _check(N.lib().zero1_sgd_step_emulated(_op(op), P, chunking, N.pointer_array(rank_grad), grad_dtype,
                                           n, master_w, momentum, lr, mu,
                                           N.pointer_array(rank_param_out), param_dtype, stream))


def ddp_buckets_launch_count(P, chunking, in_dtype, out_dtype, sgd, n, bucket_elems):
    """Kernel launches one bucketed call makes for these arguments (host only)."""
    out = ctypes.c_int64(0)
    _check(N.lib().ddp_buckets_launch_count(P, chunking, in_dtype, out_dtype, 1 if sgd else 0, n,
                                            bucket_elems, ctypes.byref(out)))
    return out.value


def zero1_sgd_step_buckets(op, P, chunking, rank_grad, grad_dtype, n, bucket_elems, master_w, momentum,
                           lr, mu, rank_param_out, param_dtype, stream=None):
    _check(N.lib().zero1_sgd_step_buckets(_op(op), P, chunking, N.pointer_array(rank_grad), grad_dtype,
                                          n, bucket_elems, master_w, momentum, lr, mu,
                                          N.pointer_array(rank_param_out), param_dtype, stream))


def reducescatter_ring_emulated(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n,
                                stream=None):
    _check(N.lib().reducescatter_ring_emulated(_op(op), P, chunking, N.pointer_array(rank_in),
                                               in_dtype, N.pointer_array(rank_out), out_dtype, n,
                                               stream))


def reducescatter_ring_buckets(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n, bucket_elems,
                               stream=None):
    _check(N.lib().reducescatter_ring_buckets(_op(op), P, chunking, N.pointer_array(rank_in), in_dtype,
                                              N.pointer_array(rank_out), out_dtype, n, bucket_elems, stream))


def allgather_ring_buckets(P, chunking, rank_buf, dtype, n, bucket_elems, stream=None):
    _check(N.lib().allgather_ring_buckets(P, chunking, N.pointer_array(rank_buf), dtype, n, bucket_elems,
                                          stream))


def allreduce_ring_stepwise_buckets(op, P, chunking, rank_buf, dtype, n, bucket_elems, sent_dev=None,
                                    stream=None):
    _check(N.lib().allreduce_ring_stepwise_buckets(_op(op), P, chunking, N.pointer_array(rank_buf), dtype, n,
                                                   bucket_elems, sent_dev, stream))


def allgather_ring_emulated(P, chunking, rank_buf, dtype, n, stream=None):
    _check(N.lib().allgather_ring_emulated(P, chunking, N.pointer_array(rank_buf), dtype, n,
                                           stream))


def allreduce_ring_stepwise(op, P, chunking, rank_buf, dtype, n, sent_dev=None, stream=None):
    _check(N.lib().allreduce_ring_stepwise(_op(op), P, chunking, N.pointer_array(rank_buf),
                                           dtype, n, sent_dev, stream))


def allreduce_tree_emulated(op, P, branching, rank_in, in_dtype, rank_out, out_dtype, n,
                            stream=None):
    _check(N.lib().allreduce_tree_emulated(_op(op), P, branching, N.pointer_array(rank_in),
                                           in_dtype, N.pointer_array(rank_out), out_dtype, n,
                                           stream))


STRATEGY_RING = 0
STRATEGY_TREE = 1
STRATEGY_CENTRALIZED = 2
_STRATEGIES = {"ring": STRATEGY_RING, "tree": STRATEGY_TREE, "centralized": STRATEGY_CENTRALIZED}


def _strategy(st):
    return st if isinstance(st, int) else _STRATEGIES[st]


def allreduce_hierarchical_emulated(op, nodes, local_ranks, local_strategy, local_param,
                                    global_strategy, global_param, rank_in, in_dtype, rank_out,
                                    out_dtype, n, stream=None):
    _check(N.lib().allreduce_hierarchical_emulated(
        _op(op), nodes, local_ranks, _strategy(local_strategy), local_param or 0,
        _strategy(global_strategy), global_param or 0, N.pointer_array(rank_in), in_dtype,
        N.pointer_array(rank_out), out_dtype, n, stream))


def allreduce_hierarchical_buckets(op, nodes, local_ranks, local_strategy, local_param,
                                   global_strategy, global_param, rank_in, in_dtype, rank_out,
                                   out_dtype, n, bucket_elems, stream=None):
    _check(N.lib().allreduce_hierarchical_buckets(
        _op(op), nodes, local_ranks, _strategy(local_strategy), local_param or 0,
        _strategy(global_strategy), global_param or 0, N.pointer_array(rank_in), in_dtype,
        N.pointer_array(rank_out), out_dtype, n, bucket_elems, stream))


TILES_DTYPE = np.dtype([("numel", "<i8"), ("first_tile", "<i4"), ("lead", "<i4")])


def ddp_multi_plan(numels, P, in_dtype, out_dtype, align_to=None):
    """Tile plan of a multi-tensor all-reduce (host only).  Returns (tiles,
    total_tiles, tile_elems); tiles is a numpy structured array in the C
    layout.  ``align_to``: one address per tensor (e.g. rank 0's inputs) to
    put the tiles on 128-byte lines of, or None."""
    numels = np.ascontiguousarray(numels, dtype=np.int64)
    tiles = np.zeros(numels.size, dtype=TILES_DTYPE)
    total = ctypes.c_int64(0)
    tile = ctypes.c_int64(0)
    _check(N.lib().ddp_multi_plan(numels.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                  numels.size, P, in_dtype, out_dtype,
                                  None if align_to is None else N.pointer_array(align_to),
                                  tiles.ctypes.data_as(ctypes.POINTER(N.TensorTiles)),
                                  ctypes.byref(total), ctypes.byref(tile)))
    return tiles, total.value, tile.value


def ddp_multi_block_map(tiles, total_tiles):
    """Block map of a multi-tensor plan (host only): entry k is the tensor
    holding tile 64 k.  Returns an int32 numpy array."""
    tiles = np.ascontiguousarray(tiles, dtype=TILES_DTYPE)
    n_blocks = ctypes.c_int64(0)
    c_tiles = tiles.ctypes.data_as(ctypes.POINTER(N.TensorTiles))
    lib = N.lib()
    _check(lib.ddp_multi_block_map(c_tiles, tiles.size, total_tiles, None, 0, ctypes.byref(n_blocks)))
    out = np.zeros(n_blocks.value, dtype=np.int32)
    _check(lib.ddp_multi_block_map(c_tiles, tiles.size, total_tiles,
                                   out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), out.size,
                                   ctypes.byref(n_blocks)))
    return out


def allreduce_multi_ring_emulated(op, P, chunking, n_tensors, tiles_dev, total_tiles, tile_elems,
                                  block_first_dev, in_ptrs_dev, in_dtype, out_ptrs_dev, out_dtype,
                                  stream=None):
    _check(N.lib().allreduce_multi_ring_emulated(_op(op), P, chunking, n_tensors, tiles_dev,
                                                 total_tiles, tile_elems, block_first_dev, in_ptrs_dev,
                                                 in_dtype, out_ptrs_dev, out_dtype, stream))


def allreduce_multi_fused_sgd(op, P, chunking, n_tensors, tiles_dev, total_tiles, tile_elems,
                              block_first_dev, in_ptrs_dev, grad_dtype, w_ptrs_dev, v_ptrs_dev, lr, mu,
                              out_ptrs_dev, out_dtype, stream=None):
    _check(N.lib().allreduce_multi_fused_sgd(_op(op), P, chunking, n_tensors, tiles_dev, total_tiles,
                                             tile_elems, block_first_dev, in_ptrs_dev, grad_dtype,
                                             w_ptrs_dev, v_ptrs_dev, lr, mu, out_ptrs_dev, out_dtype,
                                             stream))


def allreduce_multi_ring_noalloc(op, P, chunking, numels, in_ptrs, in_dtype, out_ptrs, out_dtype,
                                 stream=None):
    """The multi-tensor all-reduce from host arrays, with its tables in the
    library's per-GPU scratch area (no device allocation).  ``numels``: T
    element counts; ``in_ptrs``/``out_ptrs``: P * T device addresses,
    rank-major."""
    numels = np.ascontiguousarray(numels, dtype=np.int64)
    T = numels.size
    if len(in_ptrs) != P * T or len(out_ptrs) != P * T:
        raise ValueError(f"need {P * T} input and output pointers")
    _check(N.lib().allreduce_multi_ring_noalloc(
        _op(op), P, chunking, T, numels.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
        N.pointer_array(in_ptrs), in_dtype, N.pointer_array(out_ptrs), out_dtype, stream))


def _long_array(values):
    return (ctypes.c_int64 * len(values))(*values)


def _int_array(values):
    return (ctypes.c_int32 * len(values))(*values)


def grad_norm_multi(numels, ptrs, dtypes, workspace, workspace_bytes, norm, stream=None):
    """The global 2-norm of tensors given by host lists: T element counts,
    device addresses and dtype codes.  ``workspace`` (device, of
    grad_norm_workspace_bytes) and ``norm`` (one float) are device addresses."""
    if not len(numels) == len(ptrs) == len(dtypes):
        raise ValueError("numels, ptrs and dtypes must have one entry per tensor")
    _check(N.lib().grad_norm_multi(len(numels), _long_array(numels), N.pointer_array(ptrs), _int_array(dtypes),
                                   workspace, workspace_bytes, norm, stream))


def grad_norm_workspace_bytes(numels, ptrs, dtypes):
    """Workspace of grad_norm_multi and grad_clip_multi (host only)."""
    if not len(numels) == len(ptrs) == len(dtypes):
        raise ValueError("numels, ptrs and dtypes must have one entry per tensor")
    return _norm_bytes((len(numels), _long_array(numels), N.pointer_array(ptrs), _int_array(dtypes)))


def _norm_bytes(tensors):
    b = ctypes.c_int64(0)
    _check(N.lib().grad_norm_workspace_bytes(*tensors, ctypes.byref(b)))
    return b.value


def grad_clip_multi(numels, ptrs, dtypes, out, max_norm, norm_given, norm, workspace, workspace_bytes,
                    stream=None):
    """Clipping of tensors given by host lists (``out``: T addresses)."""
    if not len(numels) == len(ptrs) == len(dtypes) == len(out):
        raise ValueError("numels, ptrs, dtypes and out must have one entry per tensor")
    _check(N.lib().grad_clip_multi(len(numels), _long_array(numels), N.pointer_array(ptrs), _int_array(dtypes),
                                   N.pointer_array(out), max_norm, int(bool(norm_given)), norm, workspace,
                                   workspace_bytes, stream))


def allreduce_ring_norm(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n, norm, workspace,
                        workspace_bytes, stream=None):
    """``rank_out``: P addresses, or one (a single copy of the result)."""
    _check(N.lib().allreduce_ring_norm(_op(op), P, chunking, N.pointer_array(rank_in), in_dtype, len(rank_out),
                                       N.pointer_array(rank_out), out_dtype, n, norm, workspace,
                                       workspace_bytes, stream))


def allreduce_ring_norm_buckets(op, P, chunking, rank_in, in_dtype, rank_out, out_dtype, n, bucket_elems,
                                norm, workspace, workspace_bytes, stream=None):
    _check(N.lib().allreduce_ring_norm_buckets(_op(op), P, chunking, N.pointer_array(rank_in), in_dtype,
                                               len(rank_out), N.pointer_array(rank_out), out_dtype, n,
                                               bucket_elems, norm, workspace, workspace_bytes, stream))


def allreduce_norm_workspace_bytes(P, chunking, in_dtype, out_dtype, n, bucket_elems=0):
    """Workspace of the two calls above (host only); bucket_elems 0: one
    bucket."""
    b = ctypes.c_int64(0)
    _check(N.lib().allreduce_norm_workspace_bytes(P, chunking, in_dtype, out_dtype, n, bucket_elems,
                                                  ctypes.byref(b)))
    return b.value


def adamw_step_multi(numels, grads, grad_dtype, w, m, v, params, param_dtype, lr, beta1, beta2, eps,
                     weight_decay, step, step_dev=None, norm=None, max_norm=0.0, stream=None):
    """One AdamW step on tensors given by host lists of device addresses
    (``params``: T addresses or None; ``step_dev``, ``norm``: device
    addresses or None)."""
    for x in (grads, w, m, v) + ((params,) if params is not None else ()):
        if len(x) != len(numels):
            raise ValueError("every list must have one entry per tensor")
    _check(N.lib().adamw_step_multi(len(numels), _long_array(numels), N.pointer_array(grads), grad_dtype,
                                    N.pointer_array(w), N.pointer_array(m), N.pointer_array(v),
                                    N.pointer_array(params) if params is not None else None, param_dtype,
                                    lr, beta1, beta2, eps, weight_decay, step, step_dev, norm, max_norm,
                                    stream))


def _ptrs_or_none(ptrs):
    return _ptr_array(ptrs) if ptrs is not None else None


def _row_ptrs(ptrs, P):
    """P addresses or None; a P that the library refuses is left to it."""
    if ptrs is not None and len(ptrs) < P <= MAX_RANKS:
        raise ValueError(f"need {P} addresses, got {len(ptrs)}")
    return _ptrs_or_none(ptrs)


def mx4_quantize_rows(P, rank_in, in_dtype, n, rank_residual, residual_dtype, rank_codes, rank_scales, stream=None):
    """``rank_residual``: P addresses or None."""
    _check(N.lib().mx4_quantize(P, _row_ptrs(rank_in, P), in_dtype, n, _row_ptrs(rank_residual, P), residual_dtype,
                                _row_ptrs(rank_codes, P), _row_ptrs(rank_scales, P), stream))


def mx4_dequantize_rows(P, rank_codes, rank_scales, n, rank_out, out_dtype, stream=None):
    _check(N.lib().mx4_dequantize(P, _row_ptrs(rank_codes, P), _row_ptrs(rank_scales, P), n,
                                  _row_ptrs(rank_out, P), out_dtype, stream))


def allreduce_mx4_rows(op, P, rank_codes, rank_scales, n, rank_out, out_dtype, norm=None, workspace=None,
                       workspace_bytes=0, stream=None):
    """``rank_out``: P addresses, or one (a single copy of the result)."""
    _check(N.lib().allreduce_mx4(_op(op), P, _row_ptrs(rank_codes, P), _row_ptrs(rank_scales, P), n, len(rank_out),
                                 _ptrs_or_none(rank_out), out_dtype, norm, workspace, workspace_bytes, stream))


def allreduce_mx4_coded(op, P, rank_codes, rank_scales, n, out_codes, out_scales, residual=None, residual_dtype=F32,
                        norm=None, workspace=None, workspace_bytes=0, stream=None):
    """``out_codes``, ``out_scales``: P addresses each, or one."""
    if len(out_codes) != len(out_scales):
        raise ValueError("out_codes and out_scales must have one entry per row")
    _check(N.lib().allreduce_mx4_coded(_op(op), P, _row_ptrs(rank_codes, P), _row_ptrs(rank_scales, P), n,
                                       len(out_codes), _ptrs_or_none(out_codes), _ptrs_or_none(out_scales), residual,
                                       residual_dtype, norm, workspace, workspace_bytes, stream))


def allreduce_mx4_workspace_bytes(n):
    """Workspace of the two calls above with a norm (host only)."""
    b = ctypes.c_int64(0)
    _check(N.lib().allreduce_mx4_workspace_bytes(n, ctypes.byref(b)))
    return b.value


def adamw8_step_multi(numels, grads, grad_dtype, w, m, v, scales, params, param_dtype, lr, beta1, beta2, eps,
                      weight_decay, step, step_dev=None, seed=0, norm=None, max_norm=0.0, stream=None):
    """adamw_step_multi with 8-bit moments: ``m``, ``v``, ``scales`` are host
    lists of device addresses too."""
    for x in (grads, w, m, v, scales) + ((params,) if params is not None else ()):
        if len(x) != len(numels):
            raise ValueError("every list must have one entry per tensor")
    _check(N.lib().adamw8_step_multi(len(numels), _long_array(numels), N.pointer_array(grads), grad_dtype,
                                     N.pointer_array(w), N.pointer_array(m), N.pointer_array(v),
                                     N.pointer_array(scales), _ptrs_or_none(params), param_dtype, lr, beta1, beta2,
                                     eps, weight_decay, step, step_dev, seed, norm, max_norm, stream))


def adamw8_read_multi(numels, m, v, scales, m_out, v_out, out_dtype, stream=None):
    for x in (m, v, scales, m_out, v_out):
        if len(x) != len(numels):
            raise ValueError("every list must have one entry per tensor")
    _check(N.lib().adamw8_read_multi(len(numels), _long_array(numels), N.pointer_array(m), N.pointer_array(v),
                                     N.pointer_array(scales), N.pointer_array(m_out), N.pointer_array(v_out),
                                     out_dtype, stream))


def ddp_set_wg_per_cu(family, wg_per_cu):
    """Tuning knob: cap the resident workgroups per CU of one kernel family
    (a name of ``KERNEL_FAMILIES`` or its ddp_kernel_family value) for later
    launches; 0 = no cap, -1 = the built-in choice.  Results do not change."""
    if isinstance(family, str):
        if family not in N.KERNEL_FAMILIES:
            raise ValueError(f"unknown kernel family {family!r}; one of {sorted(N.KERNEL_FAMILIES)}")
        family = N.KERNEL_FAMILIES[family]
    _check(N.lib().ddp_set_wg_per_cu(family, wg_per_cu))


KERNEL_FAMILIES = dict(N.KERNEL_FAMILIES)


# --------------------------------------------------------- torch level ----

_DTYPE_CODES = {}


def torch_dtype_code(dtype):
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float32: F32, torch.bfloat16: BF16})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported element type {dtype}")
    return code


def current_stream(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _stream_for(tables):
    """Handle of the stream current on the tables' device.  The tables were
    allocated on the stream current at bind time; a launch on another stream
    is recorded on them, so that torch's allocator does not hand their memory
    out again before that launch has read it."""
    import torch
    s = torch.cuda.current_stream(tables[0].device)
    for t in tables:
        if t.device.type == "cuda":
            t.record_stream(s)
    return s.cuda_stream


def _same_device(a, b, what):
    if a[0].device != b[0].device:
        raise ValueError(f"{what}: outputs must live on the inputs' device")


def _rank_tensors(tensors, what):
    tensors = list(tensors)
    if not 1 <= len(tensors) <= MAX_RANKS:
        raise ValueError(f"{what}: need 1..{MAX_RANKS} rank tensors, got {len(tensors)}")
    t0 = tensors[0]
    device, dtype, numel = t0.get_device(), t0.dtype, t0.numel()
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{what}: tensors must live on the GPU")
        if t.get_device() != device or t.dtype != dtype or t.numel() != numel:
            raise ValueError(f"{what}: every rank needs the same device, dtype and size")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensors must be contiguous")
    return tensors


def allreduce(tensors, op="sum", chunking=None, out=None, out_dtype=None, bucket_elems=None):
    """All-reduce a list of P equal-size GPU tensors (one per rank) in the
    chunked ring order.  ``out``: list of P output tensors ("in place" when
    they are the inputs); default: new tensors of ``out_dtype`` (default the
    input dtype).  ``bucket_elems``: the tensors are flat gradient buffers
    of consecutive buckets of that many elements, each bucket all-reduced as
    its own ring (one call for all of them); None: one bucket.  Enqueued on
    the current stream; returns the outputs."""
    import torch
    tensors = _rank_tensors(tensors, "allreduce")
    P = len(tensors)
    if out is None:
        dt = out_dtype or tensors[0].dtype
        out = [torch.empty(tensors[0].shape, dtype=dt, device=tensors[0].device) for _ in range(P)]
    out = _rank_tensors(out, "allreduce out")
    if len(out) != P or out[0].numel() != tensors[0].numel():
        raise ValueError("allreduce: out must match the inputs")
    _same_device(tensors, out, "allreduce")
    if bucket_elems is not None:
        allreduce_ring_buckets(op, P, chunking or P, [t.data_ptr() for t in tensors],
                               torch_dtype_code(tensors[0].dtype), [t.data_ptr() for t in out],
                               torch_dtype_code(out[0].dtype), tensors[0].numel(), bucket_elems,
                               current_stream(tensors[0].device))
        return out
    allreduce_ring_emulated(op, P, chunking or P, [t.data_ptr() for t in tensors],
                            torch_dtype_code(tensors[0].dtype), [t.data_ptr() for t in out],
                            torch_dtype_code(out[0].dtype), tensors[0].numel(),
                            current_stream(tensors[0].device))
    return out


def allreduce_tree(tensors, op="sum", branching=2, out=None, out_dtype=None):
    """All-reduce along the b-ary tree (branching >= P-1: the centralized
    strategy).  Arguments as for ``allreduce``."""
    import torch
    tensors = _rank_tensors(tensors, "allreduce_tree")
    P = len(tensors)
    if out is None:
        dt = out_dtype or tensors[0].dtype
        out = [torch.empty(tensors[0].shape, dtype=dt, device=tensors[0].device) for _ in range(P)]
    out = _rank_tensors(out, "allreduce_tree out")
    if len(out) != P or out[0].numel() != tensors[0].numel():
        raise ValueError("allreduce_tree: out must match the inputs")
    _same_device(tensors, out, "allreduce_tree")
    allreduce_tree_emulated(op, P, branching, [t.data_ptr() for t in tensors],
                            torch_dtype_code(tensors[0].dtype), [t.data_ptr() for t in out],
                            torch_dtype_code(out[0].dtype), tensors[0].numel(),
                            current_stream(tensors[0].device))
    return out


def allreduce_hierarchical(tensors, nodes, op="sum", local=("ring", None), global_=("ring", None),
                           out=None, out_dtype=None, bucket_elems=None):
    """Two-level all-reduce: ``nodes`` nodes of len(tensors) / nodes ranks
    (node-major), each level with its own strategy, given as (name,
    parameter) with name "ring" (parameter: chunk count, None = the level's
    member count), "tree" (branching) or "centralized".  Other arguments as
    for ``allreduce`` (``bucket_elems``: every bucket its own two-level
    all-reduce)."""
    import torch
    tensors = _rank_tensors(tensors, "allreduce_hierarchical")
    P = len(tensors)
    if nodes < 1 or P % nodes:
        raise ValueError("allreduce_hierarchical: nodes must divide the rank count")
    if out is None:
        dt = out_dtype or tensors[0].dtype
        out = [torch.empty(tensors[0].shape, dtype=dt, device=tensors[0].device) for _ in range(P)]
    out = _rank_tensors(out, "allreduce_hierarchical out")
    if len(out) != P or out[0].numel() != tensors[0].numel():
        raise ValueError("allreduce_hierarchical: out must match the inputs")
    _same_device(tensors, out, "allreduce_hierarchical")
    args = (op, nodes, P // nodes, local[0], local[1], global_[0], global_[1], [t.data_ptr() for t in tensors],
            torch_dtype_code(tensors[0].dtype), [t.data_ptr() for t in out], torch_dtype_code(out[0].dtype),
            tensors[0].numel())
    if bucket_elems is not None:
        allreduce_hierarchical_buckets(*args, bucket_elems, current_stream(tensors[0].device))
    else:
        allreduce_hierarchical_emulated(*args, current_stream(tensors[0].device))
    return out


def reduce_scatter(tensors, op="sum", chunking=None, out=None, out_dtype=None, bucket_elems=None):
    """Reduce-scatter: out[owner(i)][i] receives element i's reduction
    (owner = the rank where the chunk's ring ends); every other element of
    ``out`` is left as it was.  ``bucket_elems``: every bucket of that many
    elements its own ring, as for ``allreduce``.  Returns ``out``."""
    import torch
    tensors = _rank_tensors(tensors, "reduce_scatter")
    P = len(tensors)
    if out is None:
        dt = out_dtype or tensors[0].dtype
        out = [torch.empty(tensors[0].shape, dtype=dt, device=tensors[0].device) for _ in range(P)]
    out = _rank_tensors(out, "reduce_scatter out")
    if len(out) != P or out[0].numel() != tensors[0].numel():
        raise ValueError("reduce_scatter: out must match the inputs")
    _same_device(tensors, out, "reduce_scatter")
    args = (op, P, chunking or P, [t.data_ptr() for t in tensors], torch_dtype_code(tensors[0].dtype),
            [t.data_ptr() for t in out], torch_dtype_code(out[0].dtype), tensors[0].numel())
    if bucket_elems is not None:
        reducescatter_ring_buckets(*args, bucket_elems, current_stream(tensors[0].device))
    else:
        reducescatter_ring_emulated(*args, current_stream(tensors[0].device))
    return out


def all_gather(tensors, chunking=None, bucket_elems=None):
    """All-gather in place: every rank receives each element from the rank
    that owns it.  ``bucket_elems``: every bucket of that many elements its
    own ring, as for ``allreduce``.  Returns the tensors."""
    tensors = _rank_tensors(tensors, "all_gather")
    args = (len(tensors), chunking or len(tensors), [t.data_ptr() for t in tensors],
            torch_dtype_code(tensors[0].dtype), tensors[0].numel())
    if bucket_elems is not None:
        allgather_ring_buckets(*args, bucket_elems, current_stream(tensors[0].device))
    else:
        allgather_ring_emulated(*args, current_stream(tensors[0].device))
    return tensors


def allreduce_stepwise(tensors, op="sum", chunking=None, sent=None, bucket_elems=None):
    """All-reduce fp32 rank tensors in place, one ring step per launch.
    ``sent``: optional int64 GPU tensor of P counters, increased by the
    elements each rank sends.  ``bucket_elems``: every bucket of that many
    elements its own ring, as for ``allreduce``.  Returns the tensors."""
    import torch
    tensors = _rank_tensors(tensors, "allreduce_stepwise")
    if sent is not None and (sent.dtype != torch.int64 or sent.numel() != len(tensors)
                             or sent.device != tensors[0].device or not sent.is_contiguous()):
        raise ValueError("allreduce_stepwise: sent must be a contiguous int64 tensor of P on the "
                         "tensors' device")
    args = (op, len(tensors), chunking or len(tensors), [t.data_ptr() for t in tensors],
            torch_dtype_code(tensors[0].dtype), tensors[0].numel())
    sent_ptr = sent.data_ptr() if sent is not None else None
    if bucket_elems is not None:
        allreduce_ring_stepwise_buckets(*args, bucket_elems, sent_ptr, current_stream(tensors[0].device))
    else:
        allreduce_ring_stepwise(*args, sent_ptr, current_stream(tensors[0].device))
    return tensors


class MultiAllReduce:
    """All-reduce many tensors per rank in one launch (the per-parameter
    small-message path).  Plans once for a list of shapes; ``__call__`` takes
    P lists of T tensors (rank-major) and optional P output lists."""

    def __init__(self, shapes, P, dtype, out_dtype=None, device="cuda", block_map=True):
        import torch
        self.shapes = [tuple(int(d) for d in s) for s in shapes]
        self.P = P
        self.dtype = dtype
        self.out_dtype = out_dtype or dtype
        self.device = torch.device(device)
        numels = [int(np.prod(s, dtype=np.int64)) for s in self.shapes]
        # The plan (and every table bound to it) lists the tensors smallest
        # first: the few-tile tensors, whose tiles do the least work per
        # prologue, then run while the launch fills the chip rather than in
        # its tail (measured 1.6-2% faster on the 161 ResNet-50 tensors,
        # level on the ViT-B/16 and ragged sets).  Each tensor's result does
        # not depend on the order.  plan_order[i] is the caller's index of
        # the i-th planned tensor.
        self.plan_order = sorted(range(len(numels)), key=lambda t: numels[t])
        self._planned_numels = [numels[t] for t in self.plan_order]
        # The block map lets each workgroup find its tensor with one table
        # read and a short search instead of a search over the whole plan
        # (block_map=False: the whole-plan search; same results).
        self._use_block_map = block_map
        self.tiles, self.total_tiles, self.tile_elems = ddp_multi_plan(
            self._planned_numels, P, torch_dtype_code(dtype), torch_dtype_code(self.out_dtype))
        self.tiles_dev, self.block_map, self.block_map_dev = self._upload(self.tiles, self.total_tiles)

    def _upload(self, tiles, total):
        import torch
        tiles_dev = torch.from_numpy(tiles.view(np.uint8).copy()).to(self.device)
        bmap = ddp_multi_block_map(tiles, total) if self._use_block_map else None
        bmap_dev = torch.from_numpy(bmap.copy()).to(self.device) if bmap is not None else None
        return tiles_dev, bmap, bmap_dev

    def _plan_for(self, rank_lists):
        """(tiles_dev, total_tiles, block_map_dev) for these tensors: the
        shared plan, or, when some tensor starts off a 128-byte line (a view
        into a larger buffer), a plan whose tiles follow rank 0's lines."""
        addrs = [rank_lists[0][t].data_ptr() for t in self.plan_order]
        tiles, total, _ = ddp_multi_plan(self._planned_numels, self.P, torch_dtype_code(self.dtype),
                                         torch_dtype_code(self.out_dtype), align_to=addrs)
        if not np.any(tiles["lead"]):
            return self.tiles_dev, self.total_tiles, self.block_map_dev
        tiles_dev, _, bmap_dev = self._upload(tiles, total)
        return tiles_dev, total, bmap_dev

    def _table(self, lists, dtype):
        import torch
        if len(lists) != self.P:
            raise ValueError(f"need {self.P} rank lists")
        ptrs = []
        for ts in lists:
            if len(ts) != len(self.shapes):
                raise ValueError("every rank needs one tensor per planned shape")
            for x, s in zip(ts, self.shapes):
                if tuple(x.shape) != s or x.dtype != dtype or not x.is_contiguous() \
                        or x.device != self.device:
                    raise ValueError("tensor does not match the plan")
            ptrs.extend(ts[t].data_ptr() for t in self.plan_order)
        return torch.tensor(ptrs, dtype=torch.int64).to(self.device)

    def bind(self, rank_lists, out=None):
        """Validate the tensors once and upload their pointer tables; returns
        a launcher ``run(op="sum", chunking=None)`` that enqueues the whole
        multi-tensor all-reduce with one call on the stream current at that
        call.  The launcher keeps the bound tensors (and ``out``, default:
        new tensors) alive; it always reduces those same tensors."""
        import torch
        if out is None:
            out = [[torch.empty(s, dtype=self.out_dtype, device=self.device) for s in self.shapes]
                   for _ in range(self.P)]
        tin = self._table(rank_lists, self.dtype)
        tout = self._table(out, self.out_dtype)
        tiles_dev, total, bmap_dev = self._plan_for(rank_lists)
        args = (self.P, len(self.shapes), tiles_dev.data_ptr(), total, self.tile_elems,
                bmap_dev.data_ptr() if bmap_dev is not None else None, tin.data_ptr(),
                torch_dtype_code(self.dtype), tout.data_ptr(), torch_dtype_code(self.out_dtype))
        tables = tuple(t for t in (tiles_dev, bmap_dev, tin, tout) if t is not None)

        def run(op="sum", chunking=None):
            P, T, tiles, total, tile, bmap, pin, dtin, pout, dtout = args
            allreduce_multi_ring_emulated(op, P, chunking or P, T, tiles, total, tile, bmap, pin, dtin,
                                          pout, dtout, _stream_for(tables))
            return out

        # The launcher holds raw device addresses: it must own every table
        # they point into, the tile plan included, so that it stays valid
        # after this object is dropped (``MultiAllReduce(...).bind(...)``),
        # and every tensor whose address a table holds, so that a tensor
        # the caller drops (e.g. a gradient replaced by zero_grad(set_to_none=
        # True)) is never freed and reused while the launcher can still
        # write it.  The launcher reduces exactly the tensors it was bound
        # to; new gradient tensors need a new bind().
        run.tables = tables
        run.tensors = (rank_lists, out)
        run.out = out
        return run

    def _state_table(self, ts):
        import torch
        if len(ts) != len(self.shapes):
            raise ValueError("one optimizer-state tensor per planned shape")
        for x, s in zip(ts, self.shapes):
            if tuple(x.shape) != s or x.dtype != torch.float32 or not x.is_contiguous() \
                    or x.device != self.device:
                raise ValueError("optimizer state must be contiguous float32 tensors of the planned shapes")
        return torch.tensor([ts[t].data_ptr() for t in self.plan_order], dtype=torch.int64).to(self.device)

    def bind_sgd(self, rank_grads, w, v, out=None):
        """Like bind(), for the all-reduce fused with one SGD-momentum step
        per tensor: ``w`` and ``v`` are lists of T float32 tensors (each
        parameter's master weights and momentum, updated in place); ``out``:
        optional P lists receiving the reduced gradients.  Returns
        ``run(lr, mu, op="mean", chunking=None)``."""
        tin = self._table(rank_grads, self.dtype)
        tout = self._table(out, self.out_dtype) if out is not None else None
        tw = self._state_table(w)
        tv = self._state_table(v)
        T = len(self.shapes)
        tiles_dev, total, bmap_dev = self._plan_for(rank_grads)

        tables = tuple(t for t in (tiles_dev, bmap_dev, tin, tout, tw, tv) if t is not None)

        def run(lr, mu, op="mean", chunking=None):
            allreduce_multi_fused_sgd(op, self.P, chunking or self.P, T, tiles_dev.data_ptr(), total,
                                      self.tile_elems, bmap_dev.data_ptr() if bmap_dev is not None else None,
                                      tin.data_ptr(),
                                      torch_dtype_code(self.dtype), tw.data_ptr(), tv.data_ptr(), lr, mu,
                                      tout.data_ptr() if tout is not None else None,
                                      torch_dtype_code(self.out_dtype), _stream_for(tables))
            return out

        run.tables = tables                    # owned by the launcher, as in bind()
        run.tensors = (rank_grads, w, v, out)  # every tensor the tables point to
        return run

    def __call__(self, rank_lists, op="sum", chunking=None, out=None):
        """bind() and launch once."""
        run = self.bind(rank_lists, out)
        self._last = run              # the tables must outlive the launch
        return run(op, chunking)


def zero1_sgd_step(grads, w, v, lr, mu, params, op="mean", chunking=None, bucket_elems=None):
    """ZeRO stage 1 step: reduce-scatter the rank gradients, the momentum
    step on the float32 master weights ``w`` and momentum ``v`` (updated in
    place; element i is its chunk owner's shard), and all-gather of the
    updated weights into every rank's ``params`` tensor (float32 or
    bfloat16; may be the gradient tensors themselves).  ``bucket_elems``: as
    for ``allreduce``.  Returns ``params``."""
    import torch
    grads = _rank_tensors(grads, "zero1_sgd_step")
    params = _rank_tensors(params, "zero1_sgd_step params")
    for t in (w, v):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != grads[0].numel() \
                or t.device != grads[0].device:
            raise ValueError("zero1_sgd_step: w and v must be contiguous float32 tensors of the "
                             "gradient's size on its device")
    if len(params) != len(grads) or params[0].numel() != grads[0].numel():
        raise ValueError("zero1_sgd_step: one parameter tensor per rank, of the gradient's size")
    _same_device(grads, params, "zero1_sgd_step")
    if bucket_elems is not None:
        zero1_sgd_step_buckets(op, len(grads), chunking or len(grads), [g.data_ptr() for g in grads],
                               torch_dtype_code(grads[0].dtype), grads[0].numel(), bucket_elems,
                               w.data_ptr(), v.data_ptr(), lr, mu, [p.data_ptr() for p in params],
                               torch_dtype_code(params[0].dtype), current_stream(grads[0].device))
        return params
    zero1_sgd_step_emulated(op, len(grads), chunking or len(grads), [g.data_ptr() for g in grads],
                            torch_dtype_code(grads[0].dtype), grads[0].numel(), w.data_ptr(),
                            v.data_ptr(), lr, mu, [p.data_ptr() for p in params],
                            torch_dtype_code(params[0].dtype), current_stream(grads[0].device))
    return params


def allreduce_sgd(grads, w, v, lr, mu, op="mean", chunking=None, out=None, bucket_elems=None):
    """All-reduce the rank gradients, then one SGD-momentum step on the
    float32 master weights ``w`` and momentum ``v`` (updated in place).
    ``out``: optional list of P tensors receiving the reduced gradient.
    ``bucket_elems``: as for ``allreduce`` (w and v in the same layout)."""
    import torch
    grads = _rank_tensors(grads, "allreduce_sgd")
    for t in (w, v):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != grads[0].numel() \
                or t.device != grads[0].device:
            raise ValueError("allreduce_sgd: w and v must be contiguous float32 tensors of the "
                             "gradient's size on its device")
    out_ptrs, out_code = None, F32
    if out is not None:
        out = _rank_tensors(out, "allreduce_sgd out")
        if len(out) != len(grads) or out[0].numel() != grads[0].numel():
            raise ValueError("allreduce_sgd: out must match the gradients")
        _same_device(grads, out, "allreduce_sgd")
        out_ptrs = [t.data_ptr() for t in out]
        out_code = torch_dtype_code(out[0].dtype)
    if bucket_elems is not None:
        allreduce_fused_sgd_buckets(op, len(grads), chunking or len(grads), [g.data_ptr() for g in grads],
                                    torch_dtype_code(grads[0].dtype), grads[0].numel(), bucket_elems,
                                    w.data_ptr(), v.data_ptr(), lr, mu, out_ptrs, out_code,
                                    current_stream(grads[0].device))
        return out
    allreduce_fused_sgd(op, len(grads), chunking or len(grads), [g.data_ptr() for g in grads],
                        torch_dtype_code(grads[0].dtype), grads[0].numel(), w.data_ptr(),
                        v.data_ptr(), lr, mu, out_ptrs, out_code, current_stream(grads[0].device))
    return out


# ------------------------------------------- norm, clipping, AdamW --------

def _raw_stream(index):
    """Handle of GPU ``index``'s current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _tensor_list(tensors, what, dtypes):
    import torch
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    if not tensors:
        raise ValueError(f"{what}: need at least one tensor")
    for t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {type(t).__name__} where a tensor is needed")
    device = tensors[0].device
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{what}: tensors must live on the GPU")
        if t.device != device:
            raise ValueError(f"{what}: every tensor must live on the same GPU")
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: unsupported element type {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensors must be contiguous")
    return tensors


def _scalar(x, dtype, device, what):
    """A one-element GPU tensor that a call reads."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != dtype or x.numel() != 1 or x.device != device:
        raise ValueError(f"{what} must be a tensor of one {dtype} on the gradients' device")
    return x


class _Held:
    """Tensors of a call, and their addresses as the library takes them."""

    def __init__(self, tensors, what, numels):
        self.tensors, self.what, self.numels = tuple(tensors), what, numels
        self.at = [t.data_ptr() for t in tensors]
        self.ptrs = N.pointer_array(self.at)


def _unmoved(*held):
    """Returns ``check()``, which refuses held tensors that lie elsewhere, or
    have another size, than when they were bound (0.07 us each on the host).
    It holds their storages, which keeps a held tensor's old memory from anyone
    else after ``t.data = other`` or ``t.set_()``: an address that is unchanged
    lies in the same memory."""
    import torch
    data_ptr, numel = torch.Tensor.data_ptr, torch.Tensor.numel
    tensors = sum((h.tensors for h in held), ())
    at, numels = sum((h.at for h in held), []), sum((h.numels for h in held), [])

    def check():
        if list(map(data_ptr, tensors)) == at and list(map(numel, tensors)) == numels:
            return
        for h in held:
            for k, t in enumerate(h.tensors):
                if t.data_ptr() != h.at[k] or t.numel() != h.numels[k]:
                    raise ValueError(f"{h.what}[{k}] has been given other memory or another size since it was bound "
                                     "(t.data = ..., set_, resize_): bind it again")
    check.storages = [t.untyped_storage() for t in tensors]
    return check


class MultiGrad:
    """Global norm, clipping and the AdamW step of one replica's gradients,
    many tensors per launch.  ``grads``: GPU tensors (or one), contiguous,
    float32 or bfloat16, mixed as they come.  They are checked and their
    addresses taken once; every call works on those same tensors, which this
    object keeps alive, and is enqueued on the stream current at the call.
    Gradients that are replaced by new tensors (zero_grad(set_to_none=True))
    need a new MultiGrad; a held tensor that is given other memory or another
    size (t.data = ..., set_, resize_) makes every call on it raise ValueError.
    Calls may overlap on several streams and be captured into graphs: each
    takes its own workspace from torch's allocator.  What a call writes
    (clipped gradients, w, m, v, params) it writes past autograd, as every call
    of this package does: no version counter moves, so nothing that a backward
    pass still to come has saved may be among it."""

    def __init__(self, grads):
        import torch
        self.grads = _tensor_list(grads, "MultiGrad", (torch.float32, torch.bfloat16))
        self.device = self.grads[0].device
        self._index = self.device.index
        self._new_norm = functools.partial(torch.empty_like, torch.empty((), dtype=torch.float32, device=self.device))
        self._held = _Held(self.grads, "grads", [g.numel() for g in self.grads])
        self._check = _unmoved(self._held)
        codes = [torch_dtype_code(g.dtype) for g in self.grads]
        self._list = (len(codes), _long_array(self._held.numels), self._held.ptrs, _int_array(codes))
        self._bytes = _norm_bytes(self._list)

    def _match(self, tensors, what, dtypes):
        """Tensors of the gradients' sizes, one each, on their device."""
        tensors = _tensor_list(tensors, what, dtypes)
        numels = [x.numel() for x in tensors]
        if numels != self._held.numels or tensors[0].device != self.device:
            raise ValueError(f"{what}: need one tensor of each gradient's size on its device")
        return _Held(tensors, what, numels)

    def norm(self):
        """The global 2-norm of all gradients, a float32 scalar tensor."""
        self._check()
        return self._norm()

    def _norm(self):
        import torch
        # With another GPU current, a launch on the default stream, whose
        # handle names no GPU, would go there.
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._norm()
        norm = self._new_norm()
        ws = self._workspace()
        _check(N.lib().grad_norm_multi(*self._list, ws.data_ptr() if ws is not None else None, self._bytes,
                                       norm.data_ptr(), _raw_stream(self._index)))
        return norm

    def _workspace(self):
        import torch
        return torch.empty(self._bytes, dtype=torch.uint8, device=self.device) if self._bytes else None

    def bind_clip(self, out=None):
        """Returns ``run(max_norm, norm=None)``, which scales every gradient
        by min(1, max_norm / (norm + 1e-6)), into ``out`` (one tensor per
        gradient, of its type; default: in place), and returns the norm:
        the gradients' own, computed in the same call, or the ``norm`` given
        (a float32 scalar tensor, e.g. of ``allreduce_norm``)."""
        out = self._outputs(out)
        check = self._check if out is self._held else _unmoved(self._held, out)

        def run(max_norm, norm=None):
            check()
            return self._clip(out, max_norm, norm)

        run.tensors = (self.grads, out.tensors)
        return run

    def _outputs(self, out):
        import torch
        if out is None:
            return self._held
        out = self._match(out, "clip out", (torch.float32, torch.bfloat16))
        if any(o.dtype != g.dtype for o, g in zip(out.tensors, self.grads)):
            raise ValueError("clip out: every output must have its gradient's type")
        return out

    def _clip(self, out, max_norm, norm):
        import torch
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._clip(out, max_norm, norm)
        given, ws = norm is not None, None
        if given:
            _scalar(norm, torch.float32, self.device, "norm")
        else:
            norm = self._new_norm()
            ws = self._workspace()
        _check(N.lib().grad_clip_multi(*self._list, out.ptrs, max_norm, given, norm.data_ptr(),
                                       ws.data_ptr() if ws is not None else None, self._bytes,
                                       _raw_stream(self._index)))
        return norm

    def bind_adamw(self, w, m, v, params=None):
        """Returns ``run(lr, step, betas=(0.9, 0.999), eps=1e-8,
        weight_decay=0.01, norm=None, max_norm=None)``: one AdamW step on the
        float32 master weights ``w`` and moments ``m`` and ``v`` (one tensor
        per gradient, updated in place), writing the new weights also to
        ``params`` (float32 or bfloat16) if given.  ``step``: the step's
        number from 1, an int or a tensor of one int64 on the GPU (read when
        the step runs, so that a captured step can be replayed; ``lr`` and the
        other numbers are taken at the call, so that a captured step keeps
        them).  With ``norm`` (a float32 scalar tensor) and ``max_norm`` the
        gradient is clipped on the way, and a norm that is not finite leaves
        the step out.  The gradients must all have one type."""
        bound = self._state(w, m, v, params)
        check = _unmoved(self._held, *(x for x in bound if x is not None))

        def run(lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, norm=None, max_norm=None):
            check()
            self._adamw(bound, lr, step, betas, eps, weight_decay, norm, max_norm)

        run.tensors = (self.grads, *(x.tensors if x is not None else None for x in bound))
        return run

    def _state(self, w, m, v, params):
        """w, m, v and params (or None) as a step takes them."""
        return self._float_state(w, params, (m, "m"), (v, "v"))

    def _float_state(self, w, params, *moments):
        import torch
        if any(g.dtype != self.grads[0].dtype for g in self.grads):
            raise ValueError("adamw: gradients must all have the same element type")
        w, *moments = (self._match(x, f"adamw {what}", (torch.float32,)) for x, what in ((w, "w"), *moments))
        if params is not None:
            params = self._match(params, "adamw params", (torch.float32, torch.bfloat16))
            if any(p.dtype != params.tensors[0].dtype for p in params.tensors):
                raise ValueError("adamw: params must all have the same element type")
        return (w, *moments, params)

    def bind_adamw8(self, w, moments, params=None):
        """``bind_adamw`` with the moments in 8 bits: ``moments`` is a
        ``Moments8`` of tensors of the gradients' sizes.  Returns ``run(lr, step,
        betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, norm=None,
        max_norm=None, seed=0)``.  The moments are rounded at random, by a hash
        of ``seed``, ``step`` and each element's place: the same call gives the
        same bits, and replicas that are to stay identical need the same
        seed."""
        bound = self._state8(w, moments, params)
        check = _unmoved(self._held, *(x for x in (bound[0], bound[-1]) if x is not None))
        kept = moments._kept

        def run(lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, norm=None, max_norm=None, seed=0):
            check()
            kept.check()
            self._adamw(bound, lr, step, betas, eps, weight_decay, norm, max_norm, seed)

        run.tensors = (self.grads, *(x.tensors if x is not None else None for x in bound))
        return run

    def _state8(self, w, moments, params):
        """w, m, v, scales and params (or None) as a step takes them."""
        import torch
        if not isinstance(moments, Moments8):
            raise TypeError(f"adamw8: moments must be a Moments8, not {type(moments).__name__}")
        m, v, scales = moments._held
        if m.numels != self._held.numels or moments.device != self.device:
            raise ValueError("adamw8: need moments of each gradient's size on its device")
        moments._kept.check()
        w, params = self._float_state(w, params)
        return w, m, v, scales, params

    def _adamw(self, bound, lr, step, betas, eps, weight_decay, norm, max_norm, seed=None):
        """``bound``: w, m, v and params, or with 8-bit moments w, m, v, scales
        and params, which also take the ``seed``."""
        import torch
        if (norm is None) != (max_norm is None):
            raise ValueError("adamw: norm and max_norm come together")
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._adamw(bound, lr, step, betas, eps, weight_decay, norm, max_norm, seed)
        step_dev = norm_dev = None
        if isinstance(step, torch.Tensor):
            step_dev, step = _scalar(step, torch.int64, self.device, "step").data_ptr(), 0
        if norm is not None:
            norm_dev = _scalar(norm, torch.float32, self.device, "norm").data_ptr()
        *state, params = bound
        pptrs, pcode = (params.ptrs, torch_dtype_code(params.tensors[0].dtype)) if params is not None else (None, F32)
        count, numels, ptrs, _ = self._list
        args = [count, numels, ptrs, torch_dtype_code(self.grads[0].dtype), *(x.ptrs for x in state), pptrs, pcode, lr,
                betas[0], betas[1], eps, weight_decay, step, step_dev]
        end = (norm_dev, max_norm or 0.0, _raw_stream(self._index))
        if len(state) == 3:
            _check(N.lib().adamw_step_multi(*args, *end))
        else:
            _check(N.lib().adamw8_step_multi(*args, operator.index(seed), *end))


def _present(grads, out=None):
    """The gradients that are not None (a parameter that is frozen or took
    no part has none), and their entries of ``out``."""
    import torch
    if isinstance(grads, torch.Tensor):
        return grads, out
    grads = list(grads)
    if all(g is not None for g in grads):
        return grads, out
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(grads):
            raise ValueError("clip out: need one entry per gradient")
        out = [o for g, o in zip(grads, out) if g is not None]
    return [g for g in grads if g is not None], out


def grad_norm(grads):
    """The global 2-norm of one replica's gradient tensors (float32 scalar
    tensor), entries that are None left out; see ``MultiGrad``, which a loop
    over the same tensors keeps."""
    return MultiGrad(_present(grads)[0])._norm()


def clip_grads(grads, max_norm, norm=None, out=None):
    """Scale gradient tensors so that their global 2-norm is at most
    ``max_norm``; returns the norm before.  Entries that are None are left
    out, ``out`` not looked at in their places.  See ``MultiGrad.bind_clip``."""
    grads, out = _present(grads, out)
    mg = MultiGrad(grads)
    return mg._clip(mg._outputs(out), max_norm, norm)


def adamw_step(grads, w, m, v, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, params=None,
               norm=None, max_norm=None):
    """One AdamW step on lists of tensors (or one flat buffer each); see
    ``MultiGrad.bind_adamw``."""
    mg = MultiGrad(grads)
    mg._adamw(mg._state(w, m, v, params), lr, step, betas, eps, weight_decay, norm, max_norm)


class _Kept:
    """Storages of tensors that an object keeps to itself, so that nothing but
    a resize of the storage can take their memory away: ``check()`` refuses that,
    at 0.2 us of host time per storage."""

    def __init__(self, tensors, what):
        storages = {}
        for t in tensors:
            st = t.untyped_storage()
            storages.setdefault(st.data_ptr(), st)
        self.what, self.storages = what, list(storages.values())
        self.at = [(st.data_ptr(), st.nbytes()) for st in self.storages]

    def check(self):
        if [(st.data_ptr(), st.nbytes()) for st in self.storages] != self.at:
            raise ValueError(f"{self.what}: the memory was resized since it was bound")


class Moments8:
    """The two moments of AdamW in 8 bits: for each tensor ``m`` and ``v``, a
    byte per element, and ``scales``, two bytes per block of 32 elements (lists
    of contiguous uint8 GPU tensors; adamw8_step_multi in the C header has the
    formats).  They are what a checkpoint keeps; ``Moments8(m, v, scales)`` makes
    them usable again, and ``Moments8.zeros`` new ones.  The object keeps the
    memory that the tensors have when it is made: values go in by ``copy_`` to
    them or to ``m``, ``v`` and ``scales`` of the object, and a tensor that is
    given other memory is no longer a part of it."""

    def __init__(self, m, v, scales):
        import torch
        held = []
        for x, what in ((m, "m"), (v, "v"), (scales, "scales")):
            x = [t.detach() for t in _tensor_list(x, f"Moments8 {what}", (torch.uint8,))]
            held.append(_Held(x, f"Moments8 {what}", [t.numel() for t in x]))
        numels = held[0].numels
        if held[1].numels != numels or held[2].numels != [2 * (-(-n // MX_BLOCK)) for n in numels]:
            raise ValueError("Moments8: need a byte of m and of v per element and two scale bytes per block of 32")
        self.device = held[0].tensors[0].device
        if any(h.tensors[0].device != self.device for h in held):
            raise ValueError("Moments8: every tensor must live on the same GPU")
        self._held, self.numels = held, numels
        self._kept = _Kept(sum((h.tensors for h in held), ()), "Moments8")
        self._list = (len(numels), _long_array(numels), *(h.ptrs for h in held))

    @property
    def m(self):
        return [t.detach() for t in self._held[0].tensors]

    @property
    def v(self):
        return [t.detach() for t in self._held[1].tensors]

    @property
    def scales(self):
        return [t.detach() for t in self._held[2].tensors]

    @classmethod
    def zeros(cls, tensors):
        """Moments before the first step, of the sizes of ``tensors`` (or one),
        on their device, in one allocation, each on a 128-byte line."""
        import torch
        tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
        if not tensors:
            raise ValueError("Moments8.zeros: need at least one tensor")
        numels = [t.numel() for t in tensors]
        sizes = numels + numels + [2 * (-(-n // MX_BLOCK)) for n in numels]
        padded = [-(-n // 128) * 128 for n in sizes]
        parts = torch.zeros(sum(padded), dtype=torch.uint8, device=tensors[0].device).split(padded)
        parts = [p[:n] for p, n in zip(parts, sizes)]
        T = len(tensors)
        return cls(parts[:T], parts[T:2 * T], parts[2 * T:])

    def bind_read(self, m_out, v_out):
        """Returns ``run()``, which writes the moments' values to ``m_out`` and
        ``v_out`` (one tensor of each size, all float32 or all bfloat16)."""
        bound = self._outputs(m_out, v_out)
        check = _unmoved(*bound)

        def run():
            check()
            self._read(bound)

        run.tensors = tuple(x.tensors for x in bound)
        return run

    def _outputs(self, m_out, v_out):
        import torch
        bound = []
        for x, what in ((m_out, "m_out"), (v_out, "v_out")):
            x = _tensor_list(x, f"Moments8 {what}", (torch.float32, torch.bfloat16))
            if [t.numel() for t in x] != self.numels or x[0].device != self.device:
                raise ValueError(f"Moments8 {what}: need one tensor of each moment's size on its device")
            bound.append(_Held(x, f"Moments8 {what}", self.numels))
        if len({t.dtype for h in bound for t in h.tensors}) > 1:
            raise ValueError("Moments8: outputs must all have the same element type")
        return bound

    def read(self, dtype=None):
        """The moments' values as new tensors (default float32): (list of m,
        list of v)."""
        import torch
        m, v = ([torch.empty(n, dtype=dtype or torch.float32, device=self.device) for n in self.numels]
                for _ in range(2))
        self._read(self._outputs(m, v))
        return m, v

    def _read(self, bound):
        import torch
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device.index):
                return self._read(bound)
        self._kept.check()
        _check(N.lib().adamw8_read_multi(*self._list, bound[0].ptrs, bound[1].ptrs,
                                         torch_dtype_code(bound[0].tensors[0].dtype), _raw_stream(self.device.index)))


def adamw8_step(grads, w, moments, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, params=None, norm=None,
                max_norm=None, seed=0):
    """``adamw_step`` with the moments in 8 bits (a ``Moments8``); see
    ``MultiGrad.bind_adamw8``."""
    mg = MultiGrad(grads)
    mg._adamw(mg._state8(w, moments, params), lr, step, betas, eps, weight_decay, norm, max_norm, seed)


# The workspace depends on the sizes alone; a training loop asks for the same
# ones at every step.
_norm_workspace = functools.lru_cache(maxsize=256)(allreduce_norm_workspace_bytes)


def allreduce_norm(tensors, op="sum", chunking=None, out=None, out_dtype=None, bucket_elems=None):
    """``allreduce`` that also leaves the global 2-norm of the result as one
    rank holds it; returns (outputs, norm), the norm a float32 scalar tensor.
    ``out``: P tensors, or a list of one: a single copy of the result (what
    an optimizer step on one copy of the master weights reads).  Other
    arguments as for ``allreduce``."""
    import torch
    tensors = _rank_tensors(tensors, "allreduce_norm")
    P = len(tensors)
    if out is None:
        dt = out_dtype or tensors[0].dtype
        out = [torch.empty(tensors[0].shape, dtype=dt, device=tensors[0].device) for _ in range(P)]
    out = _rank_tensors(out, "allreduce_norm out")
    x, y = tensors[0], out[0]
    n, index = x.numel(), x.get_device()
    if len(out) not in (1, P) or y.numel() != n:
        raise ValueError("allreduce_norm: out must match the inputs, P tensors or one")
    if y.get_device() != index:
        raise ValueError("allreduce_norm: outputs must live on the inputs' device")
    if bucket_elems is not None and bucket_elems < 1:
        raise ValueError("allreduce_norm: bucket_elems must be at least 1")
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return allreduce_norm(tensors, op, chunking, out, out_dtype, bucket_elems)
    icode, ocode = torch_dtype_code(x.dtype), torch_dtype_code(y.dtype)
    C = chunking or P
    need = _norm_workspace(P, C, icode, ocode, n, bucket_elems or 0)
    ws = x.new_empty(need, dtype=torch.uint8)
    norm = x.new_empty((), dtype=torch.float32)
    args = [op, P, C, [t.data_ptr() for t in tensors], icode, [t.data_ptr() for t in out], ocode, n]
    end = (norm.data_ptr(), ws.data_ptr(), need, _raw_stream(index))
    if bucket_elems is not None:
        allreduce_ring_norm_buckets(*args, bucket_elems, *end)
    else:
        allreduce_ring_norm(*args, *end)
    return out, norm
