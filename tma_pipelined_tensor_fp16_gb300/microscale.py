"""The block-scaled operators of include/tmamicro.h for torch CUDA tensors.

    Wq = mx_quantize(W, "nvfp4")                  # N x K fp16, once
    plan = MXPlan(M, N, K, format="nvfp4")
    Y = plan(mx_quantize(X, "nvfp4"), Wq)         # X . W^T, M x N
    Xt = mx_quantize(X, "nvfp4", transpose=True)  # X^T, blocked along X's columns
    Xq.values()                                   # the rounded values, fp16

Formats: ``mxfp8`` (e4m3, a power of two for every 32 values of a row), ``mxfp4``
(e2m1, a power of two for every 32) and ``nvfp4`` (e2m1, an e4m3 scale for every 16 and
one fp32 for the whole tensor, a power of two where it is found).

Argument checks and marshalling only, with the conventions of ``experts``: every operator
runs in the library's CUDA kernels, asynchronously on the current stream of the tensors'
device (or on ``stream``).
"""
import contextlib
import functools
import math

from .binding import lib
from .experts import (_call, _empty, _Handle, _out_dtype, _output, _ptr, _tensor, _torch,
                      _used_on)

MX_FORMATS = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
MX_KERNELS = {"auto": 0, "pair": 1, "single": 2}
_BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_CHUNK = {"mxfp8": 16, "mxfp4": 32, "nvfp4": 32}
_STEP = {"mxfp8": 2, "mxfp4": 3, "nvfp4": 2}    # chunks that rows are filled up to
_GROUP = {"mxfp8": 4, "mxfp4": 3, "nvfp4": 4}   # blocks of a group of scales
_WORKSPACE = 4096  # GEMM_MX_WORKSPACE_BYTES


def _format(name):
    try:
        return MX_FORMATS[name]
    except (KeyError, TypeError):
        raise ValueError("format must be one of %s" % sorted(MX_FORMATS)) from None


def _check_scale(t, format, device):
    if format != "nvfp4":
        raise ValueError("only nvfp4 has a tensor_scale")
    _tensor("tensor_scale", t, (1,), _torch().float32, device)


def _shapes(rows, K, format):
    """Shapes of the storage: codes (row blocks, chunks, 128, 16) and scales (row blocks,
    groups, 32, 4, 4)."""
    blocks = -(-rows // 128)
    step = _STEP[format]
    chunks = step * -(-K // (step * _CHUNK[format]))
    groups = -(-K // (_GROUP[format] * _BLOCK[format]))
    return (blocks, chunks, 128, 16), (blocks, groups, 32, 4, 4)


@functools.lru_cache(maxsize=512)
def _bytes(rows, K, format):
    """Offsets in an MXTensor's own memory: of the scales, behind the codes; of the tensor
    scale (16 bytes, nvfp4) and the space in which it is found; and the end.  All but the last
    are multiples of 512."""
    codes, scales = (math.prod(shape) for shape in _shapes(rows, K, format))
    end = codes + scales
    return codes, end, end + (16 + _WORKSPACE if format == "nvfp4" else 0)


class MXTensor:
    """A quantised matrix of ``rows`` x ``K``: ``codes`` and ``scales`` (uint8, in the
    storage order that include/tmamicro.h describes) and for nvfp4 ``tensor_scale`` (one
    fp32; None stands for 1)."""

    def __init__(self, rows, K, format, codes, scales, tensor_scale=None):
        torch = _torch()
        _format(format)
        if rows < 0 or K < 1:
            raise ValueError("rows must be >= 0 and K >= 1")
        shape_c, shape_s = _shapes(rows, K, format)
        _tensor("codes", codes, shape_c, torch.uint8)
        _tensor("scales", scales, shape_s, torch.uint8, codes.device)
        if tensor_scale is not None:
            _check_scale(tensor_scale, format, codes.device)
        self.rows, self.K, self.format = rows, K, format
        self.device = codes.device
        self._buffer, self._views = None, (codes, scales)
        self._given, self._found = tensor_scale, False
        self._own_scale = None

    @classmethod
    def _new(cls, rows, K, format, device, stream):
        """In one allocation, to be written by the library."""
        t = cls.__new__(cls)
        t.rows, t.K, t.format, t.device = rows, K, format, device
        t._buffer, t._views = _empty((_bytes(rows, K, format)[2],), _torch().uint8, device,
                                     stream), None
        t._given, t._found, t._own_scale = None, False, None
        return t

    def _both(self):
        if self._views is None:
            codes, scales = _shapes(self.rows, self.K, self.format)
            n, end, _ = _bytes(self.rows, self.K, self.format)
            self._views = self._buffer[:n].view(codes), self._buffer[n:end].view(scales)
        return self._views

    @property
    def codes(self):
        return self._both()[0]

    @property
    def scales(self):
        return self._both()[1]

    @property
    def tensor_scale(self):
        if not self._found:
            return self._given
        at = _bytes(self.rows, self.K, self.format)[1]
        return self._buffer[at:at + 4].view(_torch().float32)

    def _addresses(self):
        """Of the codes, the scales and the tensor scale."""
        given = None if self._given is None else self._given.data_ptr()
        if self._buffer is None:
            codes, scales = self._views
            return codes.data_ptr(), scales.data_ptr(), given
        at = self._buffer.data_ptr()
        if not at:  # no rows, no memory
            return None, None, given
        n, end, _ = _bytes(self.rows, self.K, self.format)
        return at, at + n, at + end if self._found else given

    def _parts(self):
        """The tensors that hold it."""
        return (self._views if self._buffer is None else (self._buffer,)) + (self._given,)

    @classmethod
    def from_codes(cls, codes, scales, K, format, tensor_scale=None):
        """From row-major codes (rows x K uint8 for mxfp8, rows x ceil(K / 2) for the
        others, the first of two in the low half) and row-major scales (rows x
        ceil(K / block) bytes of e8m0, e4m3 without a sign for nvfp4), as other programs
        keep them.  A set-up step."""
        torch = _torch()
        _format(format)
        rows = codes.shape[0]
        width = K if format == "mxfp8" else -(-K // 2)
        per_row = -(-K // _BLOCK[format])
        _tensor("codes", codes, (rows, width), torch.uint8)
        _tensor("scales", scales, (rows, per_row), torch.uint8, codes.device)
        (blocks, chunks, _, _), (_, groups, _, _, _) = _shapes(rows, K, format)
        c = codes.new_zeros((blocks * 128, chunks * 16))
        c[:rows, :width] = codes
        if format != "mxfp8" and K % 2:
            c[:, width - 1] &= 15
        s = scales.new_zeros((blocks * 128, groups * _GROUP[format]))
        s[:rows, :per_row] = scales
        s = torch.nn.functional.pad(s.reshape(blocks * 128, groups, -1), (0, 4 - _GROUP[format]))
        c = c.reshape(blocks, 128, chunks, 16).permute(0, 2, 1, 3).contiguous()
        s = s.reshape(blocks, 4, 32, groups, 4).permute(0, 3, 2, 1, 4).contiguous()
        return cls(rows, K, format, c, s, tensor_scale)

    def to_codes(self):
        """(codes, scales) in row-major order, as ``from_codes`` takes them."""
        blocks, chunks, _, _ = self.codes.shape
        width = self.K if self.format == "mxfp8" else -(-self.K // 2)
        c = self.codes.permute(0, 2, 1, 3).reshape(blocks * 128, chunks * 16)
        s = self.scales.permute(0, 3, 2, 1, 4)[..., :_GROUP[self.format]]
        s = s.reshape(blocks * 128, -1)
        return (c[:self.rows, :width].contiguous(),
                s[:self.rows, :-(-self.K // _BLOCK[self.format])].contiguous())

    def values(self, out=None, stream=None):
        """The values that the codes stand for (rows x K) in `out`'s type (fp16 when not
        given; fp32 holds them exactly where the tensor scale is a power of two)."""
        torch = _torch()
        dev = self.device
        dtype = torch.float32 if out is not None and out.dtype is torch.float32 else torch.float16
        V = _output("out", out, (self.rows, self.K), dtype, dev, stream)
        _call(lib().gemm_mx_values, dev, stream, self.rows, self.K, MX_FORMATS[self.format],
              *self._addresses(), 0 if dtype is torch.float32 else 1, _ptr(V))
        if stream is not None:
            _used_on(stream, *self._parts(), V)
        return V


def mx_quantize(X, format="mxfp8", transpose=False, tensor_scale=None, out=None, stream=None):
    """Round X (fp16, contiguous; its rows hold a multiple of 8 values) to `format`:
    an MXTensor of X's shape, or of X^T's with `transpose` (blocks run along X's columns).

    nvfp4: without `tensor_scale` (one fp32, 0 or larger; values beyond 2688 times it are cut
    off) it is found from X first and belongs to the result.  `out`, an MXTensor of the result's
    shape and format, is written in place and returned.  A `tensor_scale` becomes part of the
    result as it is, not as a copy."""
    torch = _torch()
    code = _format(format)
    shape = X.shape
    if len(shape) != 2:
        raise ValueError("X must be a matrix")
    _tensor("X", X, shape, torch.float16)
    dev = X.device
    rows, K = shape
    if transpose:
        rows, K = K, rows
    if K < 1:
        raise ValueError("a row must hold a value at least")
    if tensor_scale is not None:
        _check_scale(tensor_scale, format, dev)
    if out is None:
        Q = MXTensor._new(rows, K, format, dev, stream)
    else:
        Q = out
        if (Q.rows, Q.K, Q.format) != (rows, K, format) or Q.device != dev:
            raise ValueError("out must be a %s MXTensor of %d x %d on %s"
                             % (format, rows, K, dev))
    work = extra = None
    before = Q._given, Q._found
    if tensor_scale is not None:
        Q._given, Q._found = tensor_scale, False
    elif code == 2:  # nvfp4
        if Q._buffer is None:  # made by the caller: it has no room for it
            # one for all calls: a captured product finds it in place
            if Q._own_scale is None:
                Q._own_scale = _empty((1,), torch.float32, dev, stream)
            Q._given = Q._own_scale
            extra = _empty((_WORKSPACE,), torch.uint8, dev, stream)
            work = extra.data_ptr()
        else:
            Q._given, Q._found = None, True
            work = Q._buffer.data_ptr() + _bytes(rows, K, format)[1] + 16
    try:
        _call(lib().gemm_mx_quantize, dev, stream, rows, K, code, 1 if transpose else 0,
              X.data_ptr(), *Q._addresses(), work)
    except BaseException:  # its codes are the old ones: so is its scale
        Q._given, Q._found = before
        raise
    if stream is not None:
        _used_on(stream, X, *Q._parts(), extra)
    return Q


class MXPlan(_Handle):
    """C = A . B^T (M x N) of two MXTensors of one format, A of M x K and B of N x K.

    `kernel` ("auto", "pair", "single") and `split` (CTAs that share a tile's length, for
    "single") choose the kernel as in include/tmamicro.h.  Runs of a plan may overlap.
    `beside`, a plan of the same format, lends its status record: the new plan takes no device
    memory, and `device_status` of either is that of both.  A graph that captured a run needs one
    of them alive.  A plan belongs to a device: that of `beside`, or `device`, or the current one."""
    _destroy, _describe = "gemm_mx_destroy", "gemm_mx_describe"
    _status, _wait = "gemm_mx_get_device_status", "gemm_mx_set_wait"

    def __init__(self, M, N, K, format="mxfp8", out="f16", kernel="auto", split=0, beside=None,
                 device=None):
        if kernel not in MX_KERNELS:
            raise ValueError("kernel must be one of %s" % sorted(MX_KERNELS))
        code = _format(format)
        self.M, self.N, self.K, self.format = M, N, K, format
        self.dtype, out_code = _out_dtype(out)
        if beside is not None and beside.format != format:
            raise ValueError("beside is a plan of %s, not %s" % (beside.format, format))
        self.device = device if beside is None else beside.device
        with contextlib.nullcontext() if self.device is None else \
                _torch().cuda.device(self.device):
            if beside is None:
                made = lib().gemm_mx_create_plan_ex(M, N, K, code, out_code, MX_KERNELS[kernel],
                                                    split)
            else:
                made = lib().gemm_mx_create_plan_beside(beside.handle, M, N, K, out_code,
                                                        MX_KERNELS[kernel], split)
        self._own(made)

    def __call__(self, A, B, out=None, stream=None):
        for name, t, rows in (("A", A, self.M), ("B", B, self.N)):
            if not isinstance(t, MXTensor):
                raise TypeError("%s must be an MXTensor" % name)
            if t.rows != rows or t.K != self.K or t.format != self.format:
                raise ValueError("%s must be a %s MXTensor of %d x %d, not %s of %d x %d"
                                 % (name, self.format, rows, self.K, t.format, t.rows, t.K))
        dev = A.device
        if B.device != dev:
            raise ValueError("B is on %s, the other tensors on %s" % (B.device, dev))
        C = _output("out", out, (self.M, self.N), self.dtype, dev, stream)
        _call(lib().gemm_mx_run, dev, stream, self._h, *A._addresses(), *B._addresses(),
              C.data_ptr())
        if stream is not None:
            _used_on(stream, *A._parts(), *B._parts(), C)
        return C


__all__ = ["MXPlan", "MXTensor", "MX_FORMATS", "MX_KERNELS", "mx_quantize"]
