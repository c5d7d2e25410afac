"""Cases for measuring the operators around block-scaled (microscaled) products:
quantisation to 8- and 4-bit floating point with scales, the products of such
operands, the root-mean-square norm that feeds them with its gradient, and the
global gradient norm with clipping.

``listed()`` names the measured cases and ``draw(rng)`` makes more of the same
ranges; ``prepare`` makes a case's inputs, ``run`` makes one pass (``own``
selects the library's kernels or the plain form in elementary torch
operations), ``exact`` gives the same outputs in 64 bits and ``work`` the bytes
and operations that a pass cannot do without.

Formats: "mxfp8" holds e4m3 values and one power of two per 32 of them, "mxfp4"
e2m1 values and one power of two per 32, "nvfp4" e2m1 values, one e4m3 scale per
16 and one power of two for the whole tensor (1 for the norm's rows).
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
LARGEST = {"mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}
EPS = 1e-6

# The largest listed cases; drawn cases stay within them.
MAX_FLOPS = 2 * 8192 ** 3
MAX_OPERAND = 16384 * 16384
MAX_ELEMENTS = 16384 * 4096
MAX_GRADS = 2 * 16 * 2048 * 4096


def listed():
    return [
        # Activations of a training or prompt batch (16384 tokens) to 8 bits
        # and back, as a straight-through training step uses them.
        dict(name="quantize_tokens", op="quantize", rows=16384, cols=4096, format="mxfp8",
             transpose=False),
        # The same values blocked along the tokens, which the weight gradient
        # contracts: odd token count, 4 bits, the tensor's scale from its data.
        dict(name="quantize_transposed", op="quantize", rows=4001, cols=5000, format="nvfp4",
             transpose=True),
        # The headline GEMM with both operands in 4 bits.
        dict(name="product_8192", op="product", M=8192, N=8192, K=8192, format="nvfp4",
             out="f16"),
        # The ragged GEMM: no size a multiple of a tile, fp32 output.
        dict(name="product_ragged", op="product", M=4000, N=3000, K=5000, format="mxfp4",
             out="f32"),
        # The skinny GEMM: a batch of 64 tokens through 8-bit weights, bound by
        # reading them.
        dict(name="product_skinny", op="product", M=64, N=16384, K=16384, format="mxfp8",
             out="f16"),
        # One decoding token through 4-bit weights.
        dict(name="product_one", op="product", M=1, N=16384, K=16384, format="nvfp4",
             out="f16"),
        # Norm of one decoding step of 16 sequences: 0.5 MB, latency counts.
        dict(name="norm_step", op="norm", tokens=16, width=4096, residual=True, half=True,
             format="mxfp8"),
        # Norm of a training or prompt batch with the residual's sum kept, fp16
        # rows for the routed experts and 8-bit rows for block-scaled products.
        dict(name="norm_prompt", op="norm", tokens=16384, width=4096, residual=True, half=True,
             format="mxfp8"),
        # Gradient of the norm over a batch, the residual's own gradient added.
        dict(name="norm_grad_train", op="norm_grad", tokens=16384, width=4096, residual=True),
        # An odd, short batch of a wide model.
        dict(name="norm_grad_short", op="norm_grad", tokens=77, width=5120, residual=False),
        # Clipping of many small tensors: the biases, norms and small matrices
        # of a model, down to single values, fp32 and fp16 mixed.
        dict(name="clip_small", op="clip", tensors=320, largest=20000, total=0, half=0.3),
        # Clipping of the weight gradients of 16 experts, fp32: 1.07 GB.
        dict(name="clip_experts", op="clip", tensors=2, largest=16 * 2048 * 4096, total=MAX_GRADS,
             half=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(value, m):
    return max(m, value // m * m)


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "norm_grad", "clip"])
    form = rng.choice(["mxfp8", "mxfp4", "nvfp4"])
    if op == "quantize":
        cols = _mult(_log_int(rng, 64, 16384), 8)
        rows = _log_int(rng, 1, min(32768, MAX_ELEMENTS // cols))
        return dict(op=op, rows=rows, cols=cols, format=form, transpose=rng.random() < 0.5)
    if op == "product":
        K = _mult(_log_int(rng, 64, 16384), 8)
        N = _mult(_log_int(rng, 64, min(16384, MAX_OPERAND // K)), 8)
        M = _log_int(rng, 1, max(1, min(8192, MAX_FLOPS // (2 * N * K))))
        return dict(op=op, M=M, N=N, K=K, format=form, out=rng.choice(["f16", "f32"]))
    if op in ("norm", "norm_grad"):
        width = _mult(_log_int(rng, 64, 16384), 8)
        tokens = _log_int(rng, 1, min(32768, MAX_ELEMENTS // width))
        case = dict(op=op, tokens=tokens, width=width, residual=rng.random() < 0.7)
        if op == "norm":
            half = rng.random() < 0.7
            case.update(half=half, format=rng.choice(["", form]) if half else form)
        return case
    tensors = _log_int(rng, 1, 1500)
    largest = _log_int(rng, 1, min(MAX_GRADS // tensors, 1 << 24))
    return dict(op=op, tensors=tensors, largest=largest, total=0,
                half=rng.choice([0.0, 0.3, 1.0]))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _activations(g, rows, cols):
    """Rows whose channels differ in size, a few of them much larger."""
    channel = torch.exp(0.5 * _randn(g, (1, cols)))
    return (_randn(g, (rows, cols)) * channel).half()


def _operand(g, rows, K, form, scale):
    """Codes (rows x K e4m3 bytes, or rows x K/2 with the low half first) and
    scales of a quantised normal matrix, in row-major order."""
    x = (_randn(g, (rows, K)) * scale).half()
    q, s, t = _quantized(x, form, torch.float32)
    if form == "mxfp8":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE)
        c = torch.bucketize(q.abs(), level).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
        codes = c[:, 0::2] | (c[:, 1::2] << 4)
    if form == "nvfp4":
        scales = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        scales = (torch.frexp(s)[1] + 126).to(torch.uint8)
    return codes.contiguous(), scales.contiguous(), t.reshape(1)


def _lengths(case):
    """Sizes of the gradients: equal ones that make up `total`, or sizes spread
    over their logarithm up to `largest`; always the same ones for a case."""
    n = case["tensors"]
    if case["total"]:
        return [case["total"] // n] * n
    g = torch.Generator()
    g.manual_seed(n + case["largest"])
    top = math.log(case["largest"])
    return [max(1, int(v)) for v in torch.exp(torch.rand(n, generator=g) * top).tolist()]


def _types(case):
    """fp16 for the first part of the gradients, fp32 for the others."""
    n = case["tensors"]
    halves = round(case["half"] * n)
    return [torch.float16] * halves + [torch.float32] * (n - halves)


def _flat(case, dtype16, dtype32):
    """One buffer for each type, and the clipped gradients as views of them that
    start on 16 bytes, as optimisers keep them: (views, buffers)."""
    sizes, types = _lengths(case), _types(case)
    views, buffers = [None] * len(sizes), []
    for dtype, real in ((torch.float16, dtype16), (torch.float32, dtype32)):
        mine = [i for i, d in enumerate(types) if d == dtype]
        if mine:
            starts = [0]
            for i in mine:
                starts.append(starts[-1] + (sizes[i] + 7) // 8 * 8)
            buffers.append(torch.zeros(starts[-1], dtype=real, device=DEVICE))
            for i, at in zip(mine, starts):
                views[i] = buffers[-1][at:at + sizes[i]]
    return views, buffers


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case)
    if own:
        import tma_pipelined_tensor_fp16_gb300 as tg
        st["tg"] = tg
    if op == "quantize":
        st["X"] = _activations(g, case["rows"], case["cols"])
    elif op == "product":
        M, N, K, form = case["M"], case["N"], case["K"], case["format"]
        st["A"] = _operand(g, M, K, form, 1.0)
        st["B"] = _operand(g, N, K, form, 1.0 / math.sqrt(K))
        if own:
            for side in ("A", "B"):
                codes, scales, t = st[side]
                st[side] = tg.MXTensor.from_codes(codes, scales, K, form,
                                                  t if form == "nvfp4" else None)
            st["plan"] = tg.MXPlan(M, N, K, format=form, out=case["out"])
            st["C"] = torch.empty((M, N), dtype=_dtype(case["out"]), device=DEVICE)
    elif op == "norm":
        T, W = case["tokens"], case["width"]
        st["X"] = _activations(g, T, W)
        st["weight"] = (1.0 + 0.2 * _randn(g, (W,))).half()
        st["residual"] = (3.0 * _randn(g, (T, W))).half() if case["residual"] else None
    elif op == "norm_grad":
        T, W = case["tokens"], case["width"]
        st["H"] = (3.0 * _randn(g, (T, W))).half()
        st["weight"] = (1.0 + 0.2 * _randn(g, (W,))).half()
        st["dZ"] = _randn(g, (T, W)).half()
        st["dH"] = _randn(g, (T, W)).half() if case["residual"] else None
    else:
        sizes = _lengths(case)
        st["grads"] = [(_randn(g, (n,)) * 0.02).to(d) for n, d in zip(sizes, _types(case))]
        # a bound that clips, as in the steps that clipping is there for
        st["max_norm"] = 0.01 * math.sqrt(sum(sizes))
        st["out"], st["flat"] = _flat(case, torch.float16, torch.float32)
        if own:
            st["clip"] = tg.GradClip(st["grads"], out=st["out"])
    return st


def _dtype(out):
    return torch.float16 if out == "f16" else torch.float32


# -------------------------------------------------------------------- passes

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    case, tg = st["case"], st["tg"]
    op = case["op"]
    if op == "quantize":
        return [tg.mx_quantize(st["X"], case["format"], transpose=case["transpose"]).values()]
    if op == "product":
        return [st["plan"](st["A"], st["B"], st["C"])]
    if op == "norm":
        Z, H, Q = tg.rms_norm(st["X"], st["weight"], residual=st["residual"], eps=EPS,
                              half=case["half"], format=case["format"] or None)
        return dict(Z=Z, H=H if case["residual"] else None,
                    Q=Q.values() if Q is not None else None)
    if op == "norm_grad":
        return list(tg.rms_norm_grad(st["dZ"], st["H"], st["weight"], dH=st["dH"], eps=EPS))
    return [st["clip"](st["max_norm"])] + st["flat"]


def _round_e2m1(y):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    a = y.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(y.dtype)
    return torch.clamp(torch.round(a / step) * step, max=6.0) * torch.sign(y)


def _power(x, largest):
    """The least power of two p with x <= largest * p, at least 2^-126."""
    mantissa, exponent = torch.frexp(x)
    top, shift = math.frexp(largest)
    e = exponent - shift + (mantissa > top).to(exponent.dtype)
    return torch.ldexp(torch.ones_like(x), torch.where(x > 0, e, torch.full_like(e, -126)))


def _quantized(x, form, dtype, unit=False):
    """Rounded values of x along its rows, their scales, the tensor's scale (1
    with `unit`: the norm's rows, whose size is known beforehand)."""
    rows, K = x.shape
    block = BLOCK[form]
    x = x.to(dtype)
    if K % block:
        x = torch.nn.functional.pad(x, (0, block - K % block))
    x = x.reshape(rows, -1, block)
    most = x.abs().amax(-1, keepdim=True)
    t = torch.ones((), dtype=dtype, device=x.device)
    if form == "nvfp4":
        if not unit:
            t = torch.where(most.amax() > 0, _power(most.amax(), 6.0 * 448.0), t)
        s = (most / (6.0 * t)).to(torch.float8_e4m3fn).to(dtype).clamp(min=2.0 ** -9)
        q = _round_e2m1(x / (s * t))
    else:
        s = _power(most, LARGEST[form])
        q = _round_e2m1(x / s) if form == "mxfp4" else (x / s).to(torch.float8_e4m3fn).to(dtype)
    return q.reshape(rows, -1)[:, :K], s[..., 0], t


def _rounded(x, form, unit=False):
    """x through the format and back, fp16."""
    q, s, t = _quantized(x, form, torch.float32, unit)
    s = s.repeat_interleave(BLOCK[form], dim=1)[:, :q.shape[1]]
    return (q * (s * t)).half()


def _operand_values(operand, form, K):
    codes, scales, t = operand
    if form == "mxfp8":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5,
                              -2.0, -3.0, -4.0, -6.0], device=DEVICE)
        q = table[torch.stack([codes & 15, codes >> 4], dim=-1).long()].reshape(codes.shape[0], K)
    if form == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float() * t
    else:
        s = torch.ldexp(torch.ones(scales.shape, device=DEVICE), scales.int() - 127)
    return q * s.repeat_interleave(BLOCK[form], dim=1)[:, :K]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["X"].t() if case["transpose"] else st["X"]
        return [_rounded(x, case["format"])]
    if op == "product":
        a = _operand_values(st["A"], case["format"], case["K"])
        b = _operand_values(st["B"], case["format"], case["K"])
        return [(a @ b.t()).to(_dtype(case["out"]))]
    if op == "norm":
        h = st["X"].float()
        if case["residual"]:
            h = h + st["residual"].float()
        z = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["weight"].float()
        return dict(Z=z.half() if case["half"] else None,
                    H=h.half() if case["residual"] else None,
                    Q=_rounded(z, case["format"], unit=True) if case["format"] else None)
    if op == "norm_grad":
        h, dz, w = st["H"].float(), st["dZ"].float(), st["weight"].float()
        rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n, u = h * rstd, dz * w
        dx = rstd * (u - n * (u * n).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + st["dH"].float()
        return [dx.half(), (dz * n).sum(0)]
    squares = torch.stack([(t.float() * t.float()).sum(dtype=torch.float64)
                           for t in st["grads"]])
    norm = torch.sqrt(squares.sum())
    factor = torch.clamp(st["max_norm"] / (norm + EPS), max=1.0).float()
    for t, to in zip(st["grads"], st["out"]):
        to.copy_(t.float() * factor)
    return [norm.float().reshape(1)] + st["flat"]


# ---------------------------------------------------------------------- work

def _coded_bytes(rows, K, form):
    per = 1.0 if form == "mxfp8" else 0.5
    return rows * (K * per + math.ceil(K / BLOCK[form]))


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        rows, K = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"],
                                                                         case["cols"])
        # the values read, the codes written and read again, their values written
        return dict(bytes=4 * n + 2 * _coded_bytes(rows, K, case["format"]), flops=3 * n)
    if op == "product":
        M, N, K, form = case["M"], case["N"], case["K"], case["format"]
        out = 2 if case["out"] == "f16" else 4
        return dict(bytes=_coded_bytes(M, K, form) + _coded_bytes(N, K, form) + out * M * N,
                    flops=2 * M * N * K)
    if op == "norm":
        T, W = case["tokens"], case["width"]
        b = 2 * T * W * (1 + (2 if case["residual"] else 0) + (1 if case["half"] else 0)) + 2 * W
        if case["format"]:
            b += 2 * _coded_bytes(T, W, case["format"]) + 2 * T * W
        return dict(bytes=b, flops=5 * T * W)
    if op == "norm_grad":
        T, W = case["tokens"], case["width"]
        return dict(bytes=2 * T * W * (4 if case["residual"] else 3) + 6 * W, flops=10 * T * W)
    sizes = _lengths(case)
    each = [2 if d == torch.float16 else 4 for d in _types(case)]
    # every gradient read once and its clipped value written
    return dict(bytes=2 * sum(n * b for n, b in zip(sizes, each)), flops=3 * sum(sizes))


# ------------------------------------------------------------- 64-bit values

def _exact_e2m1(y):
    """The nearest level by comparison with the borders between them; a border
    itself goes to the even code."""
    a = y.abs()
    q = torch.zeros_like(a)
    for border, level, even in ((0.25, 0.5, False), (0.75, 1.0, True), (1.25, 1.5, False),
                                (1.75, 2.0, True), (2.5, 3.0, False), (3.5, 4.0, True),
                                (5.0, 6.0, False)):
        q = torch.where(a >= border if even else a > border, torch.full_like(a, level), q)
    return torch.copysign(q, y)


def _exact_e4m3(y):
    """The nearest e4m3 value: 3 bits behind the leading one, none below 2^-9."""
    e = torch.frexp(y)[1].clamp(min=-5)
    step = torch.exp2((e - 4).double())
    return torch.clamp(torch.round(y / step) * step, -448.0, 448.0)


def _exact_exponent(x, largest):
    e = torch.ceil(torch.log2(x / largest))
    e = torch.where(x > largest * torch.exp2(e), e + 1, e)
    return torch.where(x <= largest * torch.exp2(e - 1), e - 1, e)


def _exact_rounded(x, form, unit=False):
    rows, K = x.shape
    block = BLOCK[form]
    full = torch.zeros((rows, -(-K // block) * block), dtype=torch.float64, device=x.device)
    full[:, :K] = x
    b = full.view(rows, -1, block)
    most = b.abs().amax(2)
    if form == "nvfp4":
        t = 1.0 if unit else torch.exp2(_exact_exponent(most.max(), 2688.0))
        s = torch.clamp(_exact_e4m3(most / (6.0 * t)), min=2.0 ** -9) * t
    else:
        s = torch.exp2(_exact_exponent(most.clamp(min=1e-30), LARGEST[form]))
    y = b / s[:, :, None]
    y = _exact_e4m3(y) if form == "mxfp8" else _exact_e2m1(y)
    return (y * s[:, :, None]).view(rows, -1)[:, :K]


def _exact_operand(codes, scales, t, form, K):
    """Values from the bits: sign, exponent and the rest."""
    if form == "mxfp8":
        c = codes.to(torch.int32)
        sign, e, m = torch.div(c, 128, rounding_mode="floor"), (c % 128) // 8, c % 8
        v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    else:
        c = torch.empty((codes.shape[0], K), dtype=torch.int32, device=codes.device)
        c[:, 0::2] = codes.to(torch.int32) % 16
        c[:, 1::2] = codes.to(torch.int32) // 16
        sign, e, m = c // 8, (c % 8) // 2, c % 2
        v = torch.where(e > 0, (2 + m) * torch.exp2((e - 2).double()), m * 0.5)
    v = torch.where(sign > 0, -v, v)
    s = scales.to(torch.int32)
    if form == "nvfp4":
        e, m = s // 8, s % 8
        s = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
        s = s * t.double()
    else:
        s = torch.exp2((s - 127).double())
    for j in range(BLOCK[form]):  # in place: value j of every block
        part = v[:, j::BLOCK[form]]
        part *= s[:, :part.shape[1]]
    return v


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    op = case["op"]
    if op == "quantize":
        x = st["X"].double()
        return [_exact_rounded(x.t().contiguous() if case["transpose"] else x, case["format"])]
    if op == "product":
        a = _exact_operand(*st["A"], case["format"], case["K"])
        b = _exact_operand(*st["B"], case["format"], case["K"])
        return [torch.einsum("mk,nk->mn", a, b)]
    if op == "norm":
        h = st["X"].double()
        if case["residual"]:
            h += st["residual"].double()
        z = h / torch.sqrt(torch.einsum("tw,tw->t", h, h) / case["width"] + EPS)[:, None]
        z *= st["weight"].double()
        return dict(Z=z if case["half"] else None, H=h if case["residual"] else None,
                    Q=_exact_rounded(z, case["format"], unit=True) if case["format"] else None)
    if op == "norm_grad":
        h, dz, w = st["H"].double(), st["dZ"].double(), st["weight"].double()
        r = (torch.einsum("tw,tw->t", h, h) / case["width"] + EPS) ** -0.5
        dw = torch.einsum("tw,tw,t->w", dz, h, r)
        along = torch.einsum("tw,w,tw->t", dz, w, h) * r ** 3 / case["width"]
        dx = dz * w * r[:, None] - h * along[:, None]
        if case["residual"]:
            dx += st["dH"].double()
        return [dx, dw]
    norm = torch.sqrt(sum(torch.dot(t.double(), t.double()) for t in st["grads"]))
    factor = min(1.0, st["max_norm"] / (float(norm) + EPS))
    out, flat = _flat(case, torch.float64, torch.float64)
    for t, to in zip(st["grads"], out):
        to.copy_(t.double() * factor)
    return [norm.reshape(1)] + flat
