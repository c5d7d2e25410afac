"""The operators of include/tmalayer.h for torch CUDA tensors: what surrounds the products
in a layer and in its training step.

    Z, H, Q = rms_norm(X, weight, residual=R, format="mxfp8")   # H = X + R, Z = norm of H
    dX, dweight = rms_norm_grad(dZ, H, weight, dH=dH)           # dX is R's gradient, too
    clip = GradClip([dW1, dW2, dweight])
    norm = clip(1.0)                                            # the norm before clipping

Conventions are those of ``experts``.
"""
import ctypes
import functools
import math

from .binding import GemmError, last_error, lib
from .experts import _call, _empty, _output, _ptr, _tensor, _torch, _used_on
from .microscale import MXTensor, _format

_CLIP_WORKSPACE = 16384  # GEMM_CLIP_WORKSPACE_BYTES


def _matrix(name, t):
    """The shape of a contiguous fp16 CUDA matrix; raises unless `t` is one."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be a matrix (tokens x width)" % name)
    _tensor(name, t, shape, _torch().float16)
    return shape


def rms_norm(X, weight, residual=None, eps=1e-6, half=True, format=None, out=None, total=None,
             stream=None):
    """(Z, H, Q) with h = X + residual and z = h / sqrt(mean(h^2) + eps) * weight along the
    rows of X (tokens x width fp16; weight: width fp16).

    Z is z in fp16 (`out`, which may be X or residual itself unless `total` is, or a new tensor;
    None with half=False), H is h in fp16 (`total`, which may be X or residual itself, or a new
    tensor; without a residual X itself, or None where `out` has taken its place) and Q is
    z as an MXTensor of `format` (None without; nvfp4 with the tensor scale 1).  A row's
    results do not depend on the other rows, nor on how many there are."""
    torch = _torch()
    f16 = torch.float16
    shape = _matrix("X", X)
    dev = X.device
    tokens, width = shape
    _tensor("weight", weight, (width,), f16, dev)
    if residual is not None:
        _tensor("residual", residual, shape, f16, dev)
        H = _output("total", total, shape, f16, dev, stream)
        at_H = H.data_ptr()
    elif total is not None:
        raise ValueError("total is for a residual: without one it would be X")
    else:
        H, at_H = X, None
    if half:
        Z = _output("out", out, shape, f16, dev, stream)
        at_Z = Z.data_ptr()
        if out is not None and at_Z == X.data_ptr() and residual is None and tokens > 0:
            H = None
    elif out is not None:
        raise ValueError("out is not written with half=False")
    elif format is None:
        raise ValueError("half=False leaves no output without a format")
    else:
        Z = at_Z = None
    if format is None:
        Q, code, codes, scales = None, 0, None, None
    else:
        code = _format(format)
        Q = MXTensor._new(tokens, width, format, dev, stream)
        codes, scales, _ = Q._addresses()
    _call(lib().gemm_rms_norm, dev, stream, tokens, width, X.data_ptr(), _ptr(residual),
          weight.data_ptr(), eps, at_H, at_Z, code, codes, scales)
    if stream is not None:
        _used_on(stream, X, weight, residual, Z, H, *(Q._parts() if Q is not None else ()))
    return Z, H, Q


@functools.lru_cache(maxsize=256)
def _grad_workspace(tokens, width):
    """Bytes that rms_norm_grad needs."""
    size = lib().gemm_rms_norm_grad_workspace(tokens, width)
    if size < 0:
        raise GemmError(lib().gemm_last_status(), last_error())
    return size


def rms_norm_grad(dZ, H, weight, dH=None, eps=1e-6, out=None, dweight=None, stream=None):
    """(dX, dweight) of ``rms_norm`` for dZ (tokens x width fp16), its H and, with a
    residual, dH: the gradient that reaches H by its other uses.  dX (fp16; `out` may be
    dZ or dH itself) is the gradient of X and of the residual, dweight is fp32."""
    torch = _torch()
    f16 = torch.float16
    shape = _matrix("dZ", dZ)
    dev = dZ.device
    tokens, width = shape
    _tensor("H", H, shape, f16, dev)
    _tensor("weight", weight, (width,), f16, dev)
    if dH is not None:
        _tensor("dH", dH, shape, f16, dev)
    size = _grad_workspace(tokens, width)
    dX = _output("out", out, shape, f16, dev, stream)
    dw = _output("dweight", dweight, (width,), torch.float32, dev, stream)
    work = _empty((size,), torch.uint8, dev, stream)
    _call(lib().gemm_rms_norm_grad, dev, stream, tokens, width, dZ.data_ptr(), H.data_ptr(),
          weight.data_ptr(), _ptr(dH), eps, dX.data_ptr(), dw.data_ptr(), work.data_ptr())
    if stream is not None:
        _used_on(stream, dZ, H, weight, dH, dX, dw, work)
    return dX, dw


class GradClip:
    """The global norm of a list of gradients (fp32 and fp16 tensors, contiguous, any shapes,
    on one device), and clipping to it.

    ``clip(max_norm)`` writes every gradient times min(1, max_norm / (norm + eps)) into `out`
    (tensors of the same shapes and types; in place when not given) and returns the norm
    before clipping, one fp32; ``clip.norm()`` returns it alone.  The object keeps the tensors
    and a table of their addresses; a tensor whose memory has moved since is refused.  A graph
    that captured a call reads that table: the object has to live as long as the graph."""

    def __init__(self, grads, out=None):
        torch = _torch()
        self._h = None
        grads = list(grads)
        out = grads if out is None else list(out)
        if not grads:
            raise ValueError("there are no gradients")
        if len(out) != len(grads):
            raise ValueError("out must hold a tensor for each gradient")
        dev = grads[0].device
        codes = {torch.float32: 0, torch.float16: 1}
        for i, (g, o) in enumerate(zip(grads, out)):
            if g.dtype not in codes:
                raise TypeError("gradient %d must be float32 or float16, not %s" % (i, g.dtype))
            _tensor("gradient %d" % i, g, g.shape, g.dtype, dev)
            if o is not g:
                _tensor("out %d" % i, o, g.shape, g.dtype, dev)
        self.grads, self.out, self.device = grads, out, dev
        self._tensors = grads if out is grads else grads + out
        self._addresses = [t.data_ptr() for t in self._tensors]
        self._places = list(range(len(self._tensors)))
        n = len(grads)
        addresses = ctypes.c_void_p * n
        with torch.cuda.device(dev):
            self._h = lib().gemm_clip_create_plan(
                n, addresses(*self._addresses[:n]), addresses(*self._addresses[-n:]),
                (ctypes.c_int64 * n)(*[g.numel() for g in grads]),
                (ctypes.c_int * n)(*[codes[g.dtype] for g in grads]))
        if not self._h:
            raise GemmError(lib().gemm_last_status(), last_error())

    def _in_place(self, torch):
        """Whether every tensor is where it was (in one call where torch has one for its own
        graphs: 21 us for 640 tensors, one by one 37)."""
        same = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", None)
        if same is not None:
            return same(self._tensors, self._addresses, self._places)
        return [t.data_ptr() for t in self._tensors] == self._addresses

    def _run(self, fn, stream, *args):
        torch = _torch()
        if not self._in_place(torch):
            raise ValueError("a tensor's memory has moved: make a new GradClip")
        norm = _empty((1,), torch.float32, self.device, stream)
        work = _empty((_CLIP_WORKSPACE,), torch.uint8, self.device, stream)
        _call(fn, self.device, stream, self._h, *args, _ptr(norm), _ptr(work))
        if stream is not None:
            _used_on(stream, norm, work, *self._tensors)
        return norm

    def __call__(self, max_norm, eps=1e-6, stream=None):
        if not max_norm >= 0.0 or not eps >= 0.0 or math.isinf(eps):
            raise ValueError("max_norm and eps must be >= 0")
        return self._run(lib().gemm_clip_run, stream, max_norm, eps)

    def norm(self, stream=None):
        return self._run(lib().gemm_clip_norm, stream)

    def close(self):
        if self._h:
            lib().gemm_clip_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, stream=None):
    """One pass of a GradClip; it is kept by no one, so this waits for the GPU (and cannot be
    captured into a graph).  A training loop whose gradients stay where they are keeps a
    GradClip."""
    clip = GradClip(grads, out)
    norm = clip(max_norm, eps, stream)
    _torch().cuda.synchronize(clip.device)
    clip.close()
    return norm
