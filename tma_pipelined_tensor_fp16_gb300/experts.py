"""The expert-layer operators of include/tmaexperts.h for torch CUDA tensors.

A mixture-of-experts feed-forward sends each of ``tokens`` tokens to ``topk``
of ``experts`` experts.  With ``ids`` (tokens x topk, int32; negative or too
large = the slot is dropped) and routing ``weights`` (tokens x topk, float32):

    route = ExpertRoute(tokens, topk, experts).sort(ids)
    Xs = route.gather(X)                               # rows sorted by expert
    up(Xs, W1, route.offsets, H)                       # GroupedPlan "forward"
    ...                                                # activation
    down(H, W2, route.offsets, Ys)
    Y = route.combine(Ys, weights=weights)             # back to the tokens

and backwards with ``combine_grad``, the ``grad_input`` and ``grad_weight``
plans and ``gather_grad``.  ``W4Plan`` is the product for single tokens with
weights in 4 bits, dense or by expert.  ``python -m
tma_pipelined_tensor_fp16_gb300.expert_layer`` runs them together.

Argument checks and marshalling only; every operator runs in the library's CUDA
kernels, asynchronously on the current stream of the tensors' device (or on
``stream``), and writes into the tensor it is given or a new one.  A new tensor is
allocated on the stream that writes it, and with ``stream`` every tensor of the call
is marked as used there, so that its memory is not handed out again too early; as
everywhere in torch, the caller orders that stream behind the one that made the
inputs.
"""
from .binding import GEMM_OUT_F16, GEMM_OUT_F32, GemmError, _check, last_error, lib

GROUPED_OPS = {"forward": 0, "grad_input": 1, "grad_weight": 2}
W4_WEIGHTS = {"exact": 0, "rounded": 1}
GROUPED_TILES = {"auto": 0, "128x128": 1, "128x256": 2, "256x256": 3}


_modules = {}


def _torch():
    """torch, imported at the first use."""
    try:
        return _modules["torch"]
    except KeyError:
        import torch
        _modules["torch"] = torch
        return torch


def _tensor(name, t, shape, dtype, device=None):
    """Raise unless `t` is a contiguous CUDA tensor of this shape and type."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda and \
            (device is None or t.device == device):
        return t
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, device))


def _empty(shape, dtype, device, stream):
    """A new tensor, of the memory of the stream that will write it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(name, t, shape, dtype, device, stream):
    if t is None:
        return _empty(shape, dtype, device, stream)
    return _tensor(name, t, shape, dtype, device)


def _used_on(stream, *tensors):
    """Keep the memory of these tensors until the work now on `stream` is done."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _out_dtype(out):
    torch = _torch()
    if out not in ("f16", "f32"):
        raise ValueError("out must be 'f16' or 'f32'")
    return (torch.float16, GEMM_OUT_F16) if out == "f16" else (torch.float32, GEMM_OUT_F32)


def _ptr(t):
    """A tensor's address; None for no tensor (an empty one has the address 0)."""
    return None if t is None else t.data_ptr()


def _call(fn, device, stream, *args):
    """fn(*args, stream) with `device` current, on `stream` or the device's
    current stream, whose handle is returned.  Raises on an error status."""
    torch = _torch()
    index = device.index
    if torch._C._cuda_getDevice() != index:  # the tensors have set CUDA up
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    if stream is None:
        # the handle alone: a Stream object would cost as much as the launch
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = stream.cuda_stream
    status = fn(*args, handle)
    if status != 0:
        _check(status)
    return handle


class ExpertRoute:
    """The slots of one batch sorted by expert.

    ``offsets`` (experts + 1), ``order`` (tokens * topk: sorted row -> slot) and
    ``position`` (tokens x topk: slot -> sorted row) are int32 tensors, filled by
    ``sort`` or taken over by ``load``.  Dropped slots take the rows from
    ``offsets[experts]`` on.  A further ``sort`` writes the tables of the one before
    anew (so that a CUDA graph finds them in place), but never those of ``load``, which
    are the caller's.
    """

    def __init__(self, tokens, topk, experts):
        if tokens < 0 or topk < 1 or experts < 1:
            raise ValueError("tokens must be >= 0, topk and experts >= 1")
        self.tokens, self.topk, self.experts = tokens, topk, experts
        self.offsets = self.order = self.position = None
        self._home = None  # handle of the stream that the tables' memory belongs to
        self._loaded = False

    @property
    def slots(self):
        return self.tokens * self.topk

    def sort(self, ids, stream=None):
        """Sort by `ids` (tokens x topk int32); returns self."""
        torch = _torch()
        _tensor("ids", ids, (self.tokens, self.topk), torch.int32)
        dev = ids.device
        if self.offsets is None or self._loaded or self.offsets.device != dev:
            self._loaded = False
            self.offsets = _empty((self.experts + 1,), torch.int32, dev, stream)
            self.order = _empty((self.slots,), torch.int32, dev, stream)
            self.position = _empty((self.tokens, self.topk), torch.int32, dev, stream)
            self._home = None
        handle = _call(lib().gemm_expert_sort, dev, stream, self.tokens, self.topk, self.experts,
                       _ptr(ids), _ptr(self.offsets), _ptr(self.order), _ptr(self.position))
        if self._home is None:
            self._home = handle
        if handle != self._home or stream is not None:
            self._tables_used(handle, dev, stream, ids)
        return self

    def _tables_used(self, handle, dev, stream, *tensors):
        """After a launch on the stream of `handle` that is not the tables', or on the
        caller's: the tables are the route's own, so it keeps them for that stream; the
        call's tensors as always.  (The checks are the callers', for decoding's sake.)"""
        if handle != self._home:
            _used_on(stream or _torch().cuda.current_stream(dev), self.offsets, self.order,
                     self.position)
        if stream is not None:
            _used_on(stream, *tensors)

    def load(self, offsets, order, position):
        """Take over a sorted routing made elsewhere; returns self."""
        torch = _torch()
        _tensor("offsets", offsets, (self.experts + 1,), torch.int32)
        _tensor("order", order, (self.slots,), torch.int32, offsets.device)
        _tensor("position", position, (self.tokens, self.topk), torch.int32, offsets.device)
        self.offsets, self.order, self.position = offsets, order, position
        self._home = torch.cuda.current_stream(offsets.device).cuda_stream
        self._loaded = True
        return self

    def _sorted_on(self):
        if self.offsets is None:
            raise RuntimeError("the route has not been sorted: call sort() or load() first")
        return self.offsets.device

    def gather(self, X, out=None, stream=None):
        """Xs[position[t, j]] = X[t] (tokens x width fp16 -> tokens * topk x width);
        zero rows for dropped slots."""
        torch = _torch()
        dev = self._sorted_on()
        width = X.shape[-1]
        _tensor("X", X, (self.tokens, width), torch.float16, dev)
        Xs = _output("out", out, (self.slots, width), torch.float16, dev, stream)
        handle = _call(lib().gemm_expert_gather, dev, stream, self.tokens, self.topk,
                       self.experts, width, _ptr(X), _ptr(self.offsets), _ptr(self.position),
                       _ptr(Xs))
        if handle != self._home or stream is not None:
            self._tables_used(handle, dev, stream, X, Xs)
        return Xs

    def combine(self, Ys, out=None, weights=None, stream=None):
        """Y[t] = sum_j weights[t, j] * Ys[position[t, j]] over the slots that are
        not dropped (a plain sum without `weights`).  `out` is fp16 or fp32
        (fp16 when not given)."""
        dev = self._sorted_on()
        Y, code = self._combine_output(dev, Ys, out, weights, stream)
        handle = _call(lib().gemm_expert_combine, dev, stream, self.tokens, self.topk,
                       self.experts, Ys.shape[-1], _ptr(Ys), _ptr(self.offsets),
                       _ptr(self.position), _ptr(weights), code, _ptr(Y))
        if handle != self._home or stream is not None:
            self._tables_used(handle, dev, stream, Ys, weights, Y)
        return Y

    def combine_slots(self, Ys, out=None, weights=None, ids=None, stream=None):
        """As ``combine`` for rows in slot order (row t * topk + j), as W4Plan
        leaves them; needs no sort.  Slots that `ids` (tokens x topk) drops take no
        part, neither their rows nor their weights; without `ids` none is dropped."""
        dev = Ys.device
        if ids is not None:
            _tensor("ids", ids, (self.tokens, self.topk), _torch().int32, dev)
        Y, code = self._combine_output(dev, Ys, out, weights, stream)
        _call(lib().gemm_expert_combine_slots, dev, stream, self.tokens, self.topk, self.experts,
              Ys.shape[-1], _ptr(Ys), _ptr(ids), _ptr(weights), code, _ptr(Y))
        if stream is not None:
            _used_on(stream, Ys, ids, weights, Y)
        return Y

    def _combine_output(self, dev, Ys, out, weights, stream):
        """The output and its type's code; checks the operands."""
        torch = _torch()
        width = Ys.shape[-1]
        _tensor("Ys", Ys, (self.slots, width), torch.float16, dev)
        if weights is not None:
            _tensor("weights", weights, (self.tokens, self.topk), torch.float32, dev)
        dtype = torch.float32 if out is not None and out.dtype == torch.float32 else torch.float16
        Y = _output("out", out, (self.tokens, width), dtype, dev, stream)
        return Y, GEMM_OUT_F32 if dtype == torch.float32 else GEMM_OUT_F16

    def gather_grad(self, dXs, out=None, stream=None):
        """Gradient of ``gather`` with respect to X: the sum of a token's rows."""
        return self.combine(dXs, out=out, stream=stream)

    def combine_grad(self, dY, Ys, weights, out=None, dweights=None, stream=None):
        """Gradients (dYs, dweights) of the weighted ``combine`` for dY (tokens x
        width fp16).  `out` (dYs) may be Ys itself."""
        torch = _torch()
        dev = self._sorted_on()
        width = dY.shape[-1]
        _tensor("dY", dY, (self.tokens, width), torch.float16, dev)
        _tensor("Ys", Ys, (self.slots, width), torch.float16, dev)
        _tensor("weights", weights, (self.tokens, self.topk), torch.float32, dev)
        dYs = _output("out", out, (self.slots, width), torch.float16, dev, stream)
        dw = _output("dweights", dweights, (self.tokens, self.topk), torch.float32, dev, stream)
        handle = _call(lib().gemm_expert_combine_grad, dev, stream, self.tokens, self.topk,
                       self.experts, width, _ptr(dY), _ptr(Ys), _ptr(self.offsets),
                       _ptr(self.position), _ptr(weights), _ptr(dYs), _ptr(dw))
        if handle != self._home or stream is not None:
            self._tables_used(handle, dev, stream, dY, Ys, weights, dYs, dw)
        return dYs, dw


class _Handle:
    """Owner of a plan of the C library."""
    _destroy = _describe = _status = _wait = None

    def _own(self, handle):
        self._h = handle
        if not handle:
            raise GemmError(lib().gemm_last_status(), last_error())

    @property
    def handle(self):
        return self._h

    def describe(self):
        return (getattr(lib(), self._describe)(self._h) or b"").decode()

    def device_status(self):
        """GEMM_OK, or GEMM_ERR_TIMEOUT if a wait inside a kernel ran out; call
        after synchronising."""
        return getattr(lib(), self._status)(self._h)

    def set_wait(self, budget_ms=0, debug_stall=0):
        """For later runs: the bound on a wait inside the kernel (0: 2000 ms), and a
        role that is to wait in vain, for tests (see include/tmaexperts.h)."""
        status = getattr(lib(), self._wait)(self._h, budget_ms, debug_stall)
        if status != 0:
            _check(status)

    def close(self):
        if getattr(self, "_h", None):
            getattr(lib(), self._destroy)(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GroupedPlan(_Handle):
    """The experts' products over rows sorted by expert (expert e owns rows
    offsets[e] .. offsets[e + 1] - 1; B is experts x N x K):

    * ``forward``:      C[r]  = A[r] . B[e]^T      plan(A, B, offsets, C)
    * ``grad_input``:   dA[r] = dC[r] . B[e]       plan(dC, B, offsets, dA)
    * ``grad_weight``:  dB[e] = dC_e^T . A_e       plan(dC, A, offsets, dB)
    """
    _destroy, _describe = "gemm_grouped_destroy", "gemm_grouped_describe"
    _status, _wait = "gemm_grouped_get_device_status", "gemm_grouped_set_wait"

    def __init__(self, rows, N, K, experts, op="forward", out="f16", tile="auto"):
        if op not in GROUPED_OPS:
            raise ValueError("op must be one of %s" % sorted(GROUPED_OPS))
        if tile not in GROUPED_TILES:
            raise ValueError("tile must be one of %s" % sorted(GROUPED_TILES))
        self.rows, self.N, self.K, self.experts, self.op = rows, N, K, experts, op
        self.dtype, code = _out_dtype(out)
        self._own(lib().gemm_grouped_create_plan_ex(rows, N, K, experts, GROUPED_OPS[op], code,
                                                    GROUPED_TILES[tile]))

    def shapes(self):
        """Shapes of (P, Q, out)."""
        R, N, K, E = self.rows, self.N, self.K, self.experts
        return {"forward": ((R, K), (E, N, K), (R, N)),
                "grad_input": ((R, N), (E, N, K), (R, K)),
                "grad_weight": ((R, N), (R, K), (E, N, K))}[self.op]

    def __call__(self, P, Q, offsets, out=None, stream=None):
        torch = _torch()
        sp, sq, so = self.shapes()
        _tensor("P", P, sp, torch.float16)
        dev = P.device
        _tensor("Q", Q, sq, torch.float16, dev)
        _tensor("offsets", offsets, (self.experts + 1,), torch.int32, dev)
        out = _output("out", out, so, self.dtype, dev, stream)
        _call(lib().gemm_grouped_run, dev, stream, self._h, _ptr(P), _ptr(Q), _ptr(offsets),
              _ptr(out))
        if stream is not None:
            _used_on(stream, P, Q, offsets, out)
        return out


class W4Plan(_Handle):
    """Y = X . W^T with W[n, k] = scales[n, k // group] * (q[n, k] - zero) in 4 bits.

    ``packed`` is N x K/2 uint8 (the low half of byte b is q[2b], the high half
    q[2b + 1]), ``scales`` N x K/group fp16, ``zeros`` N x K/group uint8 or None
    for 8 (``w4_pack`` makes them).  With ``experts`` they are stacked, and row m
    of Y is the product of X[m // share] with the weights of expert ids[m].

    Many rows may be multiplied as fp16 matrices: with ``weights="exact"`` each weight
    as the sum of two fp16 numbers, with ``"rounded"`` rounded to one (half the
    work; the result is off by up to half a unit in the last place of each weight).
    The matrices are the plan's, so runs of a plan whose description says ``expand``
    must not overlap on the GPU (streams, threads, graph replays): one plan for each.
    """
    _destroy, _describe = "gemm_w4_destroy", "gemm_w4_describe"
    _status, _wait = "gemm_w4_get_device_status", "gemm_w4_set_wait"

    def __init__(self, M, N, K, group=128, out="f16", experts=0, share=1,
                 weights="exact"):
        if weights not in W4_WEIGHTS:
            raise ValueError("weights must be one of %s" % sorted(W4_WEIGHTS))
        self.M, self.N, self.K, self.group = M, N, K, group
        self.experts, self.share = experts, share
        self.dtype, code = _out_dtype(out)
        self._own(lib().gemm_w4_create_plan_ex(M, N, K, group, experts, share, code,
                                               W4_WEIGHTS[weights]))

    def __call__(self, X, packed, scales, out=None, zeros=None, ids=None, stream=None):
        torch = _torch()
        _tensor("X", X, (-(-self.M // self.share), self.K), torch.float16)
        dev = X.device
        lead = (self.experts,) if self.experts else ()
        groups = lead + (self.N, self.K // self.group)
        _tensor("packed", packed, lead + (self.N, self.K // 2), torch.uint8, dev)
        _tensor("scales", scales, groups, torch.float16, dev)
        if zeros is not None:
            _tensor("zeros", zeros, groups, torch.uint8, dev)
        if (ids is not None) != (self.experts > 0):
            raise ValueError("ids must be given exactly when the plan has experts")
        if ids is not None:
            if ids.numel() != self.M:
                raise ValueError("ids must hold one expert per row (%d)" % self.M)
            _tensor("ids", ids, ids.shape, torch.int32, dev)
        Y = _output("out", out, (self.M, self.N), self.dtype, dev, stream)
        _call(lib().gemm_w4_run, dev, stream, self._h, _ptr(X), _ptr(packed), _ptr(scales),
              _ptr(zeros), _ptr(ids), _ptr(Y))
        if stream is not None:
            _used_on(stream, X, packed, scales, zeros, ids, Y)
        return Y


def w4_pack(W, group=128, zeros=False):
    """Round W (... x N x K float) to 4-bit codes: (packed, scales, zeros or None)
    as W4Plan takes them.  Without `zeros` the codes are symmetric around 8 and
    the scale is the group's largest magnitude / 7; with them the group's range
    (which always holds 0) is spread over the 16 codes.  A set-up step."""
    torch = _torch()
    if W.shape[-1] % group != 0 or group not in (32, 64, 128):
        raise ValueError("K must be a multiple of group, and group 32, 64 or 128")
    w = W.float().reshape(W.shape[:-1] + (-1, group))
    if zeros:
        lo = w.amin(-1).clamp(max=0.0)
        hi = w.amax(-1).clamp(min=0.0)
        scale = ((hi - lo) / 15.0)
    else:
        scale = w.abs().amax(-1) / 7.0
    tiny = torch.finfo(torch.float16).tiny
    scales = scale.clamp(min=tiny).to(torch.float16)
    s = scales.float()[..., None]
    if zeros:
        z = (-lo / scales.float()).round().clamp(0, 15)
        q = (w / s + z[..., None]).round().clamp(0, 15)
        z = z.to(torch.uint8)
    else:
        z = None
        q = (w / s).round().clamp(-7, 7) + 8.0
    q = q.to(torch.uint8).reshape(W.shape)
    packed = q[..., 0::2] | (q[..., 1::2] << 4)
    return packed.contiguous(), scales.contiguous(), z
