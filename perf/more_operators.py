"""What the operators on compressed gradients and moments are measured on.

The step of a data-parallel job whose gradients travel in 4 bits and whose
AdamW moments are kept in 8, each operator in a plain form (elementary torch
operations) and through the package's own calls:

  quantize   P rank gradients, plus what earlier steps left over, rounded to
             microscaled 4-bit floating point; the rounding error goes back
             into the left-over; the codes are read back as values
  allreduce  P coded rank gradients decoded, added in rank order in float32,
             and written as float32, bf16 or coded again, with the 2-norm of
             what was written
  adamw8     one AdamW step of many tensors on float32 master weights and
             8-bit moments, the gradient clipped by a given norm, with a copy
             of the new weights in the model's type; the moments are read
             back as values

Formats.  A block is 32 consecutive elements of a tensor (the last one may
be shorter), with one scale byte s that stands for 2^(s - 127).

  4 bits     sign, 2 bits of exponent, 1 of mantissa: 0, .5, 1, 1.5, 2, 3, 4, 6,
             the first element of a pair in the low half of the byte.  The
             scale is the smallest that lets no element round past 6 (block
             maximum below 7 scales), the rounding to nearest, ties to even.
  m          sign, 4 bits of exponent, 3 of mantissa, up to 448; the smallest
             scale that holds the block's maximum.
  v          no sign, 5 bits of exponent, 3 of mantissa: code c stands for
             (1 + (c mod 8) / 8) * 2^((c div 8) - 31), at most 1.875; the
             smallest scale that holds the block's maximum, 0 for a block of
             zeros only, which its scale makes zero.

The moments change by less than a step of their codes, so they are rounded
at random: up with the probability of the part cut off, by 16 random bits
per value from a hash of a seed, the step's number, the tensor's number and
the element's.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 32
EPS = 1e-6          # added to the norm before the division
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # Quantisation, the smallest call: one short float32 bucket of four
        # ranks, where latency counts.
        dict(name="quantize_p4_short_f32", op="quantize", P=4, n=65536, dtype="f32", residual="f32", offset=0, scale=0.01),
        # A residual network's gradients of eight ranks in bf16, left-overs
        # in bf16 too, the rows of a bucket arena.
        dict(name="quantize_p8_bf16", op="quantize", P=8, n=25557032, dtype="bf16", residual="bf16", offset=0, scale=1e-3),
        # A quarter of a 2-billion-parameter decoder's gradient, one rank's,
        # left-overs in float32, starting inside a line.
        dict(name="quantize_long_bf16", op="quantize", P=1, n=504382464, dtype="bf16", residual="f32", offset=3, scale=1e-4),
        # All-reduce of a short bucket to every rank.
        dict(name="allreduce_p4_short", op="allreduce", P=4, n=65536, reduce="sum", out="f32", ranks=4, residual="none",
             norm=False, scale=0.01),
        # A vision transformer's gradients of eight ranks into one float32
        # copy with its norm, what the optimizer step reads next.
        dict(name="allreduce_p8_one_copy_norm", op="allreduce", P=8, n=86567656, reduce="mean", out="f32", ranks=1,
             residual="none", norm=True, scale=1e-3),
        # A residual network's gradients to all eight ranks in bf16.
        dict(name="allreduce_p8_ranks_bf16", op="allreduce", P=8, n=25557032, reduce="mean", out="bf16", ranks=8,
             residual="none", norm=False, scale=0.01),
        # Sixteen ranks, the result coded again for the way back, its error
        # kept by the owner of the result.
        dict(name="allreduce_p16_coded", op="allreduce", P=16, n=86567656, reduce="mean", out="mx4", ranks=1,
             residual="f32", norm=True, scale=1e-3),
        # AdamW, the smallest: a few small float32 tensors, nothing clipped.
        dict(name="adamw8_few_small_f32", op="adamw8", sizes="ragged", count=12, lo=1, hi=4000, shape_seed=4, dtype="f32",
             params="none", views=False, scale=0.05, clip=False, step=1, step_on_gpu=False),
        # A vision transformer's flat buffers: bf16 gradients, clipped, bf16
        # weights out, the step count on the GPU.
        dict(name="adamw8_flat_bf16", op="adamw8", sizes="flat", n=86567656, dtype="bf16", params="bf16", views=True,
             scale=1e-3, clip=True, step=1000, step_on_gpu=True),
        # Many ragged float32 tensors end to end, so that most start inside a
        # line and inside a 16-byte vector.
        dict(name="adamw8_ragged_f32", op="adamw8", sizes="ragged", count=400, lo=1000, hi=1000000, shape_seed=5, dtype="f32",
             params="none", views=True, scale=1e-2, clip=True, step=300, step_on_gpu=False),
        # The largest: a decoder's tensors as views of arenas.
        dict(name="adamw8_decoder_bf16", op="adamw8", sizes="decoder", d=2048, layers=6, vocab=50000, dtype="bf16",
             params="bf16", views=True, scale=1e-3, clip=True, step=20000, step_on_gpu=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "allreduce", "adamw8"])
    if op == "quantize":
        P = rng.choice([1, 1, 2, 4, 7, 8, 16])
        return dict(op=op, P=P, n=_log_int(rng, 1, 400000000 // P), dtype=rng.choice(["f32", "bf16"]),
                    residual=rng.choice(["none", "f32", "bf16"]), offset=rng.choice([0, 0, 1, 5, 8]),
                    scale=10.0 ** rng.uniform(-5, 0))
    if op == "allreduce":
        P = rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 12, 16])
        out = rng.choice(["f32", "bf16", "mx4"])
        return dict(op=op, P=P, n=_log_int(rng, 1, 400000000 // P), reduce=rng.choice(["sum", "mean"]), out=out,
                    ranks=rng.choice([1, P]), residual=rng.choice(["none", "f32", "bf16"]) if out == "mx4" else "none",
                    norm=rng.random() < 0.5, scale=10.0 ** rng.uniform(-5, 0))
    kind = rng.choice(["flat", "ragged", "ragged", "decoder"])
    case = dict(op=op, sizes=kind, dtype=rng.choice(["f32", "bf16"]), views=True, scale=10.0 ** rng.uniform(-4, -1))
    if kind == "flat":
        case.update(n=_log_int(rng, 1, 200000000))
    elif kind == "ragged":
        # separate tensors are few, so that all of them can be returned
        case.update(views=rng.random() < 0.5)
        case.update(count=_log_int(rng, 2, 400) if case["views"] else rng.randrange(2, 13), lo=1,
                    hi=_log_int(rng, 1000, 1000000), shape_seed=rng.randrange(1 << 30))
    else:
        case.update(d=rng.choice([256, 513, 1280, 2048]), layers=rng.randrange(1, 5), vocab=_log_int(rng, 1000, 50000))
    case.update(params=rng.choice(["none", "bf16", "f32"]), clip=rng.random() < 0.7, step=_log_int(rng, 1, 100000),
                step_on_gpu=rng.random() < 0.3)
    return case


# ---------------------------------------------------------------- inputs ----

def _numels(case):
    if case["sizes"] == "flat":
        return [case["n"]]
    if case["sizes"] == "ragged":
        rng = random.Random(case["shape_seed"])
        return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["count"])]
    d, ffn, vocab = case["d"], 7 * case["d"], case["vocab"]
    block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, ffn * d, ffn, d * ffn, d]
    return [vocab * d] + block * case["layers"] + [d, d, vocab * d]


def _blocks(n):
    return -(-n // BLOCK)


def _rows(P, n, dtype, offset=0):
    """P rows of n elements, each 4 KiB-aligned and then `offset` elements."""
    pad = 4096 // (4 if dtype == "f32" else 2)
    base = torch.empty(P, -(-(n + offset) // pad) * pad + pad, dtype=TYPES[dtype], device=DEV)
    return [base[r, offset:offset + n] for r in range(P)]


def _lay_out(numels, dtype, views):
    """Empty tensors of these sizes and what holds them: end to end in one
    flat buffer, or one allocation each."""
    if not views:
        tensors = [torch.empty(n, dtype=dtype, device=DEV) for n in numels]
        return tensors, tensors
    flat = torch.empty(sum(numels), dtype=dtype, device=DEV)
    return list(flat.split(numels)), [flat]


def _normal(held, std, gen):
    for x in held:
        x.copy_(torch.randn(x.numel(), device=DEV, generator=gen).mul_(std))


def _coded_rows(rows):
    """What the ranks hold after a quantisation: [blocks * 16] codes and
    [blocks] scales, uint8, of each row."""
    coded = []
    for x in rows:
        q, s = _round4(_to_blocks(x.float()))
        coded.append((_pack4(q), s))
    return coded


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "quantize":
        s["rows"] = _rows(case["P"], case["n"], case["dtype"], case["offset"])
        _normal(s["rows"], case["scale"], gen)
        s["left"] = None
        if case["residual"] != "none":
            # what a rounding left: up to a sixth of a block's maximum
            s["left"] = _rows(case["P"], case["n"], case["residual"], case["offset"])
            _normal(s["left"], 0.15 * case["scale"], gen)
        return s
    if case["op"] == "allreduce":
        # one row at a time: the ranks' gradients are not kept
        rows = (torch.randn(case["n"], device=DEV, generator=gen).mul_(case["scale"]) for _ in range(case["P"]))
        s["coded"] = _coded_rows(rows)
        s["left"] = None
        if case["residual"] != "none":
            s["left"] = _rows(1, case["n"], case["residual"])[0]
            _normal([s["left"]], 0.15 * case["scale"], gen)
        s["out"] = None if case["out"] == "mx4" else _rows(case["ranks"], case["n"], case["out"])
        return s
    numels = _numels(case)
    s["grads"], s["held"] = _lay_out(numels, TYPES[case["dtype"]], case["views"])
    _normal(s["held"], case["scale"], gen)
    # gradients of different layers differ in size by some powers of two
    rng = random.Random(int(seed))
    for g in s["grads"]:
        g.mul_(2.0 ** rng.randrange(-3, 4))
    s["w"], s["w_held"] = _lay_out(numels, torch.float32, case["views"])
    _normal(s["w_held"], 0.02, gen)
    s["p"] = s["p_held"] = None
    if case["params"] != "none":
        s["p"], s["p_held"] = _lay_out(numels, TYPES[case["params"]], case["views"])
    # moments as earlier steps leave them; none before the first
    s["m"], s["m_held"] = _lay_out(numels, torch.uint8, case["views"])
    s["v"], s["v_held"] = _lay_out(numels, torch.uint8, case["views"])
    s["scales"], s["scales_held"] = _lay_out([2 * _blocks(n) for n in numels], torch.uint8, case["views"])
    if case["step"] > 1:
        for t, n in enumerate(numels):
            m = torch.randn(n, device=DEV, generator=gen).mul_(0.3 * case["scale"])
            v = torch.randn(n, device=DEV, generator=gen).mul_(case["scale"]).square_()
            _store_moments(m, v, s["m"][t], s["v"][t], s["scales"][t], _random_bits(n, int(seed) + t))
    else:
        for x in s["m_held"] + s["v_held"] + s["scales_held"]:
            x.zero_()
    s["step"] = torch.full((1,), case["step"], dtype=torch.int64, device=DEV) if case["step_on_gpu"] else case["step"]
    s["norm"] = _square_sum(s["held"]).sqrt().float() if case["clip"] else None
    # where the moments are read back to
    s["m_out"], s["m_out_held"] = _lay_out(numels, torch.bfloat16, case["views"])
    s["v_out"], s["v_out_held"] = _lay_out(numels, torch.bfloat16, case["views"])
    return s


HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
MAX_NORM = 1.0      # of the clipped AdamW cases
SR_SEED = 20240229  # of the moments' rounding


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import gradient_all_reduce_allreduce_amd as ddp
        if case["op"] == "allreduce":
            s["mx"] = [ddp.Mx4(codes, scales, case["n"]) for codes, scales in s["coded"]]
        if case["op"] == "adamw8":
            # the handles that a training loop makes once for its tensors
            moments = ddp.Moments8(s["m"], s["v"], s["scales"])
            s["call"] = ddp.MultiGrad(s["grads"]).bind_adamw8(s["w"], moments, params=s["p"])
            s["read"] = moments.bind_read(s["m_out"], s["v_out"])
    return s


# ------------------------------------------------------------------ runs ----

def run(s):
    case = s["case"]
    return {"quantize": _run_quantize, "allreduce": _run_allreduce, "adamw8": _run_adamw8}[case["op"]](s, case)


def _square_sum(held):
    """The sum of the squares of all elements: squares in float32, their sum
    in float64 (float32 sums of 10^9 squares lose digits)."""
    return torch.stack([x.float().square().sum(dtype=torch.float64) for x in held]).sum()


def _power2(e):
    """2^e as float32 for whole e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_blocks(x):
    """[..., n] as [..., blocks, 32], zeros behind the end."""
    n = x.shape[-1]
    return torch.nn.functional.pad(x, (0, _blocks(n) * BLOCK - n)).unflatten(-1, (-1, BLOCK))


def _from_blocks(x, n):
    return x.flatten(-2)[..., :n]


def _round4(t):
    """[..., blocks, 32] float32 to the nearest levels, in scales; and the
    scale bytes."""
    fraction, exponent = torch.frexp(t.abs().amax(-1))      # fraction in [.5, 1)
    k = torch.clamp(exponent - 1 + (fraction >= 0.875).int() - 2, min=-126)
    x = t / _power2(k).unsqueeze(-1)
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.clamp((a / step).round_() * step, max=6.0), x), (k + 127).to(torch.uint8)


def _pack4(q):
    """Levels [..., blocks, 32] as bytes [..., blocks * 16]."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += torch.signbit(q).to(torch.uint8) << 3
    return (code[..., 0::2] + (code[..., 1::2] << 4)).flatten(-2)


def _values4(codes, scales, n):
    """What coded rows [..., blocks * 16], [..., blocks] stand for, float32 [..., n]."""
    levels = torch.tensor(LEVELS + [-x for x in LEVELS], device=codes.device)
    pairs = torch.stack([levels[(codes & 15).int()], levels[(codes >> 4).int()]], -1)
    values = pairs.flatten(-2).unflatten(-1, (-1, BLOCK)) * _power2(scales.int() - 127).unsqueeze(-1)
    return _from_blocks(values, n)


def _run_quantize(s, case):
    dtype = TYPES[case["dtype"]]
    if own:
        import gradient_all_reduce_allreduce_amd as ddp
        coded = ddp.mx4_quantize(s["rows"], residual=s["left"])
        values = ddp.mx4_dequantize(coded, dtype=dtype)
        return {"values": values, "left": s["left"]}
    t = torch.stack(s["rows"]).float()
    if s["left"] is not None:
        t += torch.stack(s["left"])
    q, scales = _round4(_to_blocks(t))
    codes = _pack4(q)
    del q
    values = _values4(codes, scales, case["n"])
    if s["left"] is not None:
        [left.copy_(x) for left, x in zip(s["left"], t.sub_(values))]
    return {"values": list(values.to(dtype)), "left": s["left"]}


def _run_allreduce(s, case):
    P, n, ranks = case["P"], case["n"], case["ranks"]
    if own:
        import gradient_all_reduce_allreduce_amd as ddp
        call = ddp.allreduce_mx4_norm if case["norm"] else ddp.allreduce_mx4
        if case["out"] == "mx4":
            out = call(s["mx"], case["reduce"], out=[ddp.Mx4.empty(n, DEV) for _ in range(ranks)], residual=s["left"])
        else:
            out = call(s["mx"], case["reduce"], out=s["out"])
        out, norm = out if case["norm"] else (out, None)
        if case["out"] == "mx4":
            out = ddp.mx4_dequantize(out, dtype=torch.bfloat16)
        return {"out": out, "left": s["left"], "norm": norm}
    g = _values4(torch.stack([c for c, _ in s["coded"]]), torch.stack([x for _, x in s["coded"]]), n)
    g = g.sum(0) if case["reduce"] == "sum" else g.mean(0)
    if case["out"] == "mx4":
        if s["left"] is not None:
            g += s["left"]
        q, scales = _round4(_to_blocks(g))
        codes = _pack4(q).unsqueeze(0).repeat(ranks, 1)
        values = _values4(codes, scales.unsqueeze(0).repeat(ranks, 1), n)
        if s["left"] is not None:
            s["left"].copy_(g.sub_(values[0]))
        out = list(values.bfloat16())
    else:
        g = g.to(TYPES[case["out"]])
        out = [o.copy_(g) for o in s["out"]]
    return {"out": out, "left": s["left"], "norm": _square_sum(out[:1]).sqrt().float() if case["norm"] else None}


M32 = 0xffffffff


def _mix(x):
    """A bijection of 32 bits, with the fractions of the roots of 3 and 5."""
    x ^= x >> 16
    x = x * 0xBB67AE85 & M32
    x ^= x >> 15
    x = x * 0x3C6EF373 & M32
    return x ^ x >> 16


def _key(seed, step, tensor, piece):
    """The key of a tensor's random bits at a step; pieces of 2^30 elements."""
    h = 0
    for word in (seed & M32, seed >> 32 & M32, step & M32, step >> 32 & M32, tensor, piece):
        h = _mix((h ^ word) + 0x9E3779B9 & M32)
    return h


def _random_bits(n, key):
    """32 random bits for each element, as int64."""
    x = torch.arange(n, dtype=torch.int64, device=DEV).mul_(0x9E3779B9).add_(key).bitwise_and_(M32)
    x ^= x >> 15
    x.mul_(0xBB67AE85).bitwise_and_(M32)
    return x ^ x >> 16


def _at_random(x, lowest, bits):
    """x >= 0 rounded to 4 significant bits (fewer below 2^lowest), up with
    the probability of what is cut off; 16 random bits."""
    step = _power2(torch.clamp(torch.frexp(x).exponent - 1, min=lowest) - 3)
    return torch.floor(x / step + (bits.float() + 0.5) / 65536) * step


def _store_moments(m, v, m_codes, v_codes, scales, bits):
    """Round the moments [n] and write their codes."""
    n = m.numel()
    low, high = _to_blocks(bits & 0xffff), _to_blocks(bits >> 16)
    m, v = _to_blocks(m), _to_blocks(v)
    fraction, exponent = torch.frexp(m.abs().amax(-1))
    k = torch.clamp(exponent - 9 + (fraction > 0.875).int(), min=-126)
    q = _at_random(m.abs() / _power2(k).unsqueeze(-1), -6, low)
    m_codes.copy_(_from_blocks(torch.copysign(q, m), n).to(torch.float8_e4m3fn).view(torch.uint8))
    fraction, exponent = torch.frexp(v.amax(-1))
    e = torch.clamp(exponent - 1 + (fraction > 0.9375).int(), min=-95)
    q = torch.clamp(_at_random(v / _power2(e).unsqueeze(-1), -31, high), min=2.0 ** -31)
    fraction_q, exponent_q = torch.frexp(q)
    v_codes.copy_(_from_blocks((exponent_q + 30) * 8 + (fraction_q * 16).int() - 8, n))
    scales.view(-1, 2)[:, 0] = (k + 127).to(torch.uint8)
    scales.view(-1, 2)[:, 1] = torch.where(fraction > 0, e + 127, 0).to(torch.uint8)


def _moments(m_codes, v_codes, scales):
    """What the codes stand for, float32 [n]."""
    n = m_codes.numel()
    scale = (scales.view(-1, 2).int() << 23).view(torch.float32)
    m = _to_blocks(m_codes).view(torch.float8_e4m3fn).float() * scale[:, :1]
    v = _to_blocks(v_codes).int()
    v = ((v << 20) + (96 << 23)).view(torch.float32) * scale[:, 1:]
    return _from_blocks(m, n), _from_blocks(v, n)


def _adamw8_plain(t, g, w, m_codes, v_codes, scales, p, m_out, v_out, c, step, fixes, h):
    """The step on one tensor; weights and moments are updated in place."""
    g = g.float() if c is None else g.float() * c
    m, v = _moments(m_codes, v_codes, scales)
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + g * g * (1 - h["beta2"])
    update = (m / fixes[0]) / ((v / fixes[1]).sqrt_() + h["eps"])
    w.mul_(1 - h["lr"] * h["weight_decay"]).sub_(update * h["lr"])
    if p is not None:
        p.copy_(w)
    _store_moments(m, v, m_codes, v_codes, scales, _random_bits(g.numel(), _key(SR_SEED, step, t, 0)))
    m, v = _moments(m_codes, v_codes, scales)
    m_out.copy_(m)
    v_out.copy_(v)


def _run_adamw8(s, case):
    if own:
        s["call"](HYPER["lr"], s["step"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"],
                  weight_decay=HYPER["weight_decay"], norm=s["norm"], max_norm=MAX_NORM if case["clip"] else None,
                  seed=SR_SEED)
        s["read"]()
    else:
        c = torch.clamp(MAX_NORM / (s["norm"] + EPS), max=1.0) if case["clip"] else None
        fixes = [1 - HYPER[b] ** (s["step"].double() if case["step_on_gpu"] else s["step"]) for b in ("beta1", "beta2")]
        fixes = [x.float() if torch.is_tensor(x) else x for x in fixes]
        params = s["p"] or [None] * len(s["grads"])
        [_adamw8_plain(t, *tensors, c, case["step"], fixes, HYPER) for t, tensors in
         enumerate(zip(s["grads"], s["w"], s["m"], s["v"], s["scales"], params, s["m_out"], s["v_out"]))]
    return {"w": s["w_held"], "m": s["m_out_held"], "v": s["v_out_held"], "params": s["p_held"]}


# ---------------------------------------------------------- work and truth ----

def work(case):
    size = {"f32": 4, "bf16": 2, "none": 0}
    if case["op"] == "quantize":
        coded = _blocks(case["n"]) * 17
        each = size[case["dtype"]] + 2 * size[case["residual"]] + size[case["dtype"]]
        return {"bytes": case["P"] * (case["n"] * each + 2 * coded), "flops": case["P"] * case["n"] * 6}
    if case["op"] == "allreduce":
        n, coded = case["n"], _blocks(case["n"]) * 17
        if case["out"] == "mx4":    # written coded, then read back as bf16
            out = case["ranks"] * (2 * coded + 2 * n) + 2 * n * size[case["residual"]]
        else:
            out = case["ranks"] * n * size[case["out"]]
        return {"bytes": case["P"] * coded + out + 4 * case["norm"], "flops": n * (2 * case["P"] + 2)}
    n = sum(_numels(case))
    blocks = sum(_blocks(k) for k in _numels(case))
    # gradient, weights, moments in and out; then the moments again and their values
    return {"bytes": n * (size[case["dtype"]] + 8 + 4 + size[case["params"]]) + 4 * blocks + 6 * n + 2 * blocks,
            "flops": 40 * n}


def _two64(e):
    """2^e in float64 for whole e, from its bits: a power function may be off
    by its last digit, and ties have to stay ties."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _levels64(x):
    """x, in scales, to the level nearest to it; of two the one whose place in
    the list is even."""
    a = x.abs()
    place = torch.zeros_like(a, dtype=torch.int64)
    for j in range(7):
        middle = (LEVELS[j] + LEVELS[j + 1]) / 2
        place += (a > middle) if j % 2 == 0 else (a >= middle)
    return torch.tensor(LEVELS, dtype=torch.float64, device=x.device)[place] * torch.sign(x)


def _nearest64(t):
    """A float64 row [n] as its 4-bit codes stand for it."""
    out = torch.empty_like(t)
    span = BLOCK << 20      # some blocks at a time
    for at in range(0, t.numel(), span):
        x = t[at:at + span]
        b = torch.zeros(-(-x.numel() // BLOCK) * BLOCK, dtype=torch.float64, device=t.device)
        b[:x.numel()] = x
        b = b.view(-1, BLOCK)
        top = b.abs().max(1, keepdim=True).values
        # the smallest power of two with top / scale < 7
        k = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -140) / 7)) + 1
        k += (top >= 7 * _two64(k)).double()
        k -= (top < 7 * _two64(k - 1)).double()
        scale = _two64(torch.clamp(k, min=-126))
        out[at:at + span] = (_levels64(b / scale) * scale).view(-1)[:x.numel()]
    return out


def _decode64(codes, scales, n):
    """A coded row's values in float64, byte by byte."""
    c = torch.empty(codes.numel() * 2, dtype=torch.float64, device=codes.device)
    table = torch.tensor([v * f for f in (1, -1) for v in LEVELS], dtype=torch.float64, device=codes.device)
    c[0::2] = table[(codes % 16).long()]
    c[1::2] = table[(codes // 16).long()]
    return (c.view(-1, BLOCK) * _two64(scales.double() - 127).unsqueeze(1)).view(-1)[:n]


def exact(case, seed):
    """What run() returns, from the definitions in float64.  The sum that is
    quantised (gradient and left-over) is by definition a float32 value."""
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        values, left = [], []
        for r in range(case["P"]):
            t = s["rows"][r].double()
            if s["left"] is not None:
                t = (t + s["left"][r].double()).float().double()
            q = _nearest64(t)
            values.append(q)
            left.append(t - q)
        return {"values": values, "left": left if s["left"] is not None else None}
    if case["op"] == "allreduce":
        g = torch.zeros(case["n"], dtype=torch.float64, device=DEV)
        for codes, scales in s["coded"]:
            g += _decode64(codes, scales, case["n"])
        if case["reduce"] == "mean":
            g /= case["P"]
        left = None
        if case["out"] == "mx4":
            t = g.float().double()
            if s["left"] is not None:
                t = (t + s["left"].double()).float().double()
            g = _nearest64(t)
            left = t - g if s["left"] is not None else None
        return {"out": [g] * case["ranks"], "left": left,
                "norm": torch.linalg.vector_norm(g) if case["norm"] else None}
    c = 1.0
    if case["clip"]:
        norm = sum(float((x.double() ** 2).sum()) for x in s["held"]) ** 0.5
        c = min(1.0, MAX_NORM / (norm + EPS))
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], case["step"]
    want = {"w": [], "m": [], "v": []}
    for i, g in enumerate(s["grads"]):
        n = g.numel()
        m, v = _decode_moments64(s["m"][i], s["v"][i], s["scales"][i])
        g = g.double() * c
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        w = s["w"][i].double() * (1 - HYPER["lr"] * HYPER["weight_decay"])
        w -= HYPER["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + HYPER["eps"])
        bits = _random_bits(n, _key(SR_SEED, t, i, 0)).double()
        upper = torch.floor(bits / 65536)
        # m: the top level of a scale is 448, from 2^-6 down the steps are equal
        want["m"].append(_random64(m, 448.0, 0, -6, bits - 65536 * upper))
        # v: the top level is 1.875, and nothing in a block that is not all zero goes below 2^-31
        want["v"].append(_random64(v, 1.875, 2.0 ** -31, -31, upper))
        want["w"].append(w)
    if case["views"]:
        want = {k: [torch.cat(x)] for k, x in want.items()}
    if case["params"] != "none":
        want["params"] = want["w"]
    return want


def _decode_moments64(m_codes, v_codes, scales):
    """8-bit moments' values in float64, field by field."""
    def each(byte):
        return torch.repeat_interleave(scales[byte::2].double(), BLOCK)[:m_codes.numel()]
    c = m_codes.double()
    sign = 1 - 2 * torch.floor(c / 128)
    c = c % 128
    field, part = torch.floor(c / 8), c % 8
    m = torch.where(field > 0, (1 + part / 8) * _two64(field - 7), part * 2.0 ** -9) * sign
    c = v_codes.double()
    v = (1 + c % 8 / 8) * _two64(torch.floor(c / 8) - 31)
    v_scale = each(1)
    return m * _two64(each(0) - 127), torch.where(v_scale > 0, v * _two64(v_scale - 127), 0.0)


def _random64(x, top, least, lowest, bits):
    """x rounded at random to codes whose top level is `top` scales."""
    n = x.numel()
    b = torch.zeros(2, -(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    b[0, :n], b[1, :n] = x, bits
    b, r = b.view(2, -1, BLOCK)
    most = b.abs().max(1, keepdim=True).values
    k = torch.ceil(torch.log2(torch.clamp(most, min=2.0 ** -140) / top))
    k += (most > top * _two64(k)).double()
    k -= (most <= top * _two64(k - 1)).double()
    scale = _two64(torch.clamp(k, min=-126 if least == 0 else -95))
    a = b.abs() / scale
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(a, min=2.0 ** -200))), min=lowest)
    e += (a >= _two64(e + 1)).double()
    e -= ((a < _two64(e)) & (e > lowest)).double()
    step = _two64(e - 3)
    q = torch.clamp(torch.floor(a / step + (r + 0.5) / 65536) * step, min=least)
    return (torch.where(most > 0, q, 0.0) * torch.sign(torch.where(b == 0, 1.0, b)) * scale).view(-1)[:n]
