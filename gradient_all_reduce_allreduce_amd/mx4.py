"""Gradients in microscaled 4-bit floating point: quantisation with a
residual, reading back, and the all-reduce of coded gradients (the C header's
mx4_quantize, mx4_dequantize, allreduce_mx4 and allreduce_mx4_coded, which
hold the format and the rules).

A step of a data-parallel job whose gradients travel in 4 bits::

    coded = plan.alloc_mx4(P)                       # one Mx4 per rank
    left = plan.alloc_arena(P, torch.bfloat16).zero_()
    left = [left[r, :plan.total] for r in range(P)]
    ddp.mx4_quantize(rows, residual=left, out=coded)
    _, norm = ddp.allreduce_mx4_norm(coded, "mean", out=[grad])
"""

from . import api
from ._native import DDP_MX_BLOCK as BLOCK


def _blocks(numel):
    return -(-numel // BLOCK)


class Mx4:
    """One rank's coded gradient of ``numel`` elements: ``codes``, 16 bytes per
    block of 32 elements, on a 16-byte line, and ``scales``, a byte per block
    (contiguous uint8 GPU tensors).  The object keeps the memory that they have
    when it is made; a tensor that is given other memory is no longer a part of
    it."""

    __slots__ = ("numel", "device", "_parts", "_kept", "codes_at", "scales_at")

    def __init__(self, codes, scales, numel):
        import torch
        if numel < 0:
            raise ValueError(f"Mx4: numel = {numel} is negative")
        for x, what, size in ((codes, "codes", 16 * _blocks(numel)), (scales, "scales", _blocks(numel))):
            if not isinstance(x, torch.Tensor) or x.dtype != torch.uint8:
                raise TypeError(f"Mx4: {what} must be a uint8 tensor")
            if not x.is_cuda:
                raise ValueError(f"Mx4: {what} must live on the GPU")
            if not x.is_contiguous() or x.numel() != size:
                raise ValueError(f"Mx4: {what} must be contiguous and hold {size} bytes for {numel} elements")
        if codes.device != scales.device:
            raise ValueError("Mx4: codes and scales must live on the same GPU")
        codes, scales = codes.detach().view(-1), scales.detach().view(-1)
        self._set(int(numel), codes, 0, scales, 0, api._Kept((codes, scales), "Mx4"))

    def _set(self, numel, codes, codes_from, scales, scales_from, kept):
        self.numel, self.device, self._kept = numel, codes.device, kept
        self._parts = (codes, codes_from, scales, scales_from)
        self.codes_at = codes.data_ptr() + codes_from
        self.scales_at = scales.data_ptr() + scales_from
        return self

    @classmethod
    def rows(cls, P, numel, device="cuda"):
        """Room for P rows of ``numel`` elements in one allocation, each on a
        4 KiB line and no two a power of two apart: a list of P Mx4."""
        import torch
        if numel < 0:
            raise ValueError(f"Mx4: numel = {numel} is negative")
        blocks = _blocks(numel)
        stride = -(-17 * blocks // 4096) * 4096 + 4096
        memory = torch.empty(P * stride, dtype=torch.uint8, device=device)
        kept = api._Kept((memory,), "Mx4")
        return [cls.__new__(cls)._set(numel, memory, r * stride, memory, r * stride + 16 * blocks, kept)
                for r in range(P)]

    @classmethod
    def empty(cls, numel, device="cuda"):
        """Room for ``numel`` elements."""
        return cls.rows(1, numel, device)[0]

    @property
    def codes(self):
        x, at = self._parts[:2]
        return x[at:at + 16 * _blocks(self.numel)]

    @property
    def scales(self):
        x, at = self._parts[2:]
        return x[at:at + _blocks(self.numel)]

    def narrow(self, start, length):
        """The elements ``start`` .. ``start + length - 1`` as an Mx4 in the
        same memory, e.g. one bucket: ``start`` a multiple of 32, and
        ``length`` too unless it reaches the end."""
        if not 0 <= start <= start + length <= self.numel:
            raise ValueError(f"Mx4.narrow: elements {start} to {start + length} of {self.numel}")
        if start % BLOCK or (length % BLOCK and start + length != self.numel):
            raise ValueError("Mx4.narrow: must begin and end at blocks of 32 elements")
        b = start // BLOCK
        codes, c, scales, s = self._parts
        return Mx4.__new__(Mx4)._set(length, codes, c + 16 * b, scales, s + b, self._kept)


def _coded_rows(coded, what):
    """Checked rows and their addresses."""
    coded = list(coded)
    if not 1 <= len(coded) <= api.MAX_RANKS:
        raise ValueError(f"{what}: need 1..{api.MAX_RANKS} coded rows, got {len(coded)}")
    kept = None
    for c in coded:
        if not isinstance(c, Mx4):
            raise TypeError(f"{what}: {type(c).__name__} where an Mx4 is needed")
        if c.numel != coded[0].numel or c.device != coded[0].device:
            raise ValueError(f"{what}: every row needs the same device and size")
        if c._kept is not kept:
            kept = c._kept
            kept.check()
    return coded, [c.codes_at for c in coded], [c.scales_at for c in coded]


def _new_rows(P, n, dtype, device):
    """P tensors of n elements in one allocation, each on a 4 KiB line."""
    import torch
    line = 4096 // (2 if dtype == torch.bfloat16 else 4)
    return list(torch.empty(P, -(-n // line) * line + line, dtype=dtype, device=device)[:, :n].unbind(0))


def _residual_tensors(residual, like, what):
    residual = api._rank_tensors(residual, f"{what} residual")
    if len(residual) != len(like) or residual[0].numel() != like[0].numel() \
            or residual[0].get_device() != like[0].get_device():
        raise ValueError(f"{what}: residual must match the gradients, one tensor per rank")
    return residual


def mx4_quantize(tensors, residual=None, out=None):
    """Code P rank gradients (equal-size float32 or bfloat16 GPU tensors) in
    4 bits; returns a list of P ``Mx4`` (``out``, or new ones).  ``residual``:
    P float32 or bfloat16 tensors, zero before the first step, which are added
    to the gradients first and receive what the rounding leaves.  Enqueued on
    the current stream."""
    import torch
    tensors = api._rank_tensors(tensors, "mx4_quantize")
    x = tensors[0]
    n, index = x.numel(), x.get_device()
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return mx4_quantize(tensors, residual, out)
    left, lcode = None, api.F32
    if residual is not None:
        residual = _residual_tensors(residual, tensors, "mx4_quantize")
        left, lcode = [t.data_ptr() for t in residual], api.torch_dtype_code(residual[0].dtype)
    out, codes, scales = _coded_rows(out if out is not None else Mx4.rows(len(tensors), n, x.device), "mx4_quantize out")
    if len(out) != len(tensors) or out[0].numel != n or out[0].device != x.device:
        raise ValueError("mx4_quantize: out must match the gradients, one Mx4 per rank")
    api.mx4_quantize_rows(len(tensors), [t.data_ptr() for t in tensors], api.torch_dtype_code(x.dtype), n, left, lcode,
                          codes, scales, api._raw_stream(index))
    return out


def mx4_dequantize(coded, out=None, dtype=None):
    """The values of P coded rows; returns a list of P tensors (``out``, or new
    ones of ``dtype``, default float32)."""
    import torch
    coded, codes, scales = _coded_rows(coded, "mx4_dequantize")
    n, device = coded[0].numel, coded[0].device
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return mx4_dequantize(coded, out, dtype)
    out = api._rank_tensors(out, "mx4_dequantize out") if out is not None \
        else _new_rows(len(coded), n, dtype or torch.float32, device)
    if len(out) != len(coded) or out[0].numel() != n or out[0].get_device() != device.index:
        raise ValueError("mx4_dequantize: out must match the coded rows, one tensor per rank")
    api.mx4_dequantize_rows(len(coded), codes, scales, n, [t.data_ptr() for t in out],
                            api.torch_dtype_code(out[0].dtype), api._raw_stream(device.index))
    return out


def allreduce_mx4(coded, op="sum", out=None, out_dtype=None, residual=None):
    """All-reduce P coded rank gradients: their values added in float32 in rank
    order, divided by P for "mean".  ``out``: P tensors or one (a single copy,
    in a list or by itself), float32 or bfloat16; or P ``Mx4`` or one, and the
    result is coded again (rows may be the inputs), with ``residual`` the owner's
    error from step to step (one float32 or bfloat16 tensor) if given.  Default: P
    new tensors of ``out_dtype`` (default float32).  Enqueued on the current
    stream; returns the list of outputs."""
    return _allreduce(coded, op, out, out_dtype, residual, False)[0]


def allreduce_mx4_norm(coded, op="sum", out=None, out_dtype=None, residual=None):
    """``allreduce_mx4`` that also leaves the global 2-norm of the result as
    one rank holds it; returns (outputs, norm), the norm a float32 scalar
    tensor."""
    return _allreduce(coded, op, out, out_dtype, residual, True)


def _allreduce(coded, op, out, out_dtype, residual, with_norm):
    import torch
    coded, codes, scales = _coded_rows(coded, "allreduce_mx4")
    P, n, device = len(coded), coded[0].numel, coded[0].device
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _allreduce(coded, op, out, out_dtype, residual, with_norm)
    if out is None:
        out = _new_rows(P, n, out_dtype or torch.float32, device)
    elif isinstance(out, Mx4) or (isinstance(out, torch.Tensor) and out.dim() < 2 and not n == 1 < out.numel()):
        out = [out]     # (a longer tensor where n is 1 holds rows of one element)
    else:
        out = list(out)
    again = any(isinstance(o, Mx4) for o in out)
    if again:
        out, out_codes, out_scales = _coded_rows(out, "allreduce_mx4 out")
        size, where = out[0].numel, out[0].device.index
    else:
        out = api._rank_tensors(out, "allreduce_mx4 out")
        size, where = out[0].numel(), out[0].get_device()
    if len(out) not in (1, P) or size != n or where != index:
        raise ValueError("allreduce_mx4: out must match the inputs, P rows or one")
    left, lcode = None, api.F32
    if residual is not None:
        if not again:
            raise ValueError("allreduce_mx4: a residual belongs to a coded result")
        residual, = api._rank_tensors([residual], "allreduce_mx4 residual")
        if residual.numel() != n or residual.get_device() != index:
            raise ValueError("allreduce_mx4: residual must be one tensor of the rows' size on their device")
        left, lcode = residual.data_ptr(), api.torch_dtype_code(residual.dtype)
    norm, end = None, (None, None, 0)
    if with_norm:
        norm = torch.empty((), dtype=torch.float32, device=device)
        need = api.allreduce_mx4_workspace_bytes(n)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        end = (norm.data_ptr(), ws.data_ptr(), need)
    stream = api._raw_stream(index)
    if again:
        api.allreduce_mx4_coded(op, P, codes, scales, n, out_codes, out_scales, left, lcode, *end, stream)
    else:
        api.allreduce_mx4_rows(op, P, codes, scales, n, [t.data_ptr() for t in out],
                               api.torch_dtype_code(out[0].dtype), *end, stream)
    return out, norm
