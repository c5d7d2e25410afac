"""The block-scaled formats in numpy, 64 bits: rounding, decoding, storage order.

Everything here follows from the formats' definition (include/tmamicro.h) with
arithmetic that is exact in 64 bits, so codes and scales are compared bit for bit.
"""
import numpy as np

BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
LARGEST = {"mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The value of each byte (127 and 255: NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(b & 128, -v, v)
    v[[127, 255]] = np.nan
    return v


def nearest(x, levels):
    """Index of the level nearest to |x| (ties: the even index; above the last: it)."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(levels, a), 1, len(levels) - 1)
    lo = hi - 1
    up, down = levels[hi] - a, a - levels[lo]
    pick_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def power_of_two(a, largest):
    """Least e with a <= largest * 2^e, at least -127 (a = 0: -127)."""
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(np.where(a > 0, a, 1.0) / largest))
    e = np.where(a > largest * 2.0 ** e, e + 1, e)
    e = np.where(a <= largest * 2.0 ** (e - 1), e - 1, e)
    return np.where(a > 0, np.maximum(e, -127.0), -127.0)


def tensor_scale(x):
    finite = np.abs(x[np.isfinite(x)])
    most = finite.max() if finite.size else 0.0
    return 1.0 if most == 0 else float(2.0 ** power_of_two(most, 2688.0))


def quantize(x, format, t=None):
    """(codes rows x K, one to an entry; scales rows x blocks, bytes; t) of 64-bit x."""
    rows, K = x.shape
    block = BLOCK[format]
    pad = -K % block
    b = np.pad(x.astype(np.float64), ((0, 0), (0, pad))).reshape(rows, -1, block)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    a = np.abs(b).max(-1) if rows else np.zeros(b.shape[:2])
    if format == "nvfp4":
        t = tensor_scale(x) if t is None else t
        levels = e4m3_values()[:127]
        scales = np.maximum(nearest(a / (6.0 * t), levels), 1)
        s = levels[scales] * t
        scales = np.where(bad, 127, scales)
    else:
        t = 1.0
        e = power_of_two(a, LARGEST[format])
        s = 2.0 ** e
        scales = np.where(bad, 255, e + 127)
    y = b / s[..., None]
    levels = e4m3_values()[:127] if format == "mxfp8" else E2M1
    sign = np.where(np.signbit(y), 128 if format == "mxfp8" else 8, 0)
    codes = (nearest(y, levels) | sign).reshape(rows, -1)[:, :K]
    return codes.astype(np.uint8), scales.astype(np.uint8), t


def values(codes, scales, format, t=1.0):
    """The 64-bit values of codes (one to an entry) and scale bytes."""
    K = codes.shape[1]
    if format == "mxfp8":
        q = e4m3_values()[codes]
    else:
        q = np.where(codes & 8, -E2M1[codes & 7], E2M1[codes & 7])
    if format == "nvfp4":
        s = e4m3_values()[scales] * t
    else:
        s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return q * np.repeat(s, BLOCK[format], axis=1)[:, :K]


def pack(codes, format):
    """Codes one to an entry -> row-major bytes."""
    if format == "mxfp8":
        return np.ascontiguousarray(codes)
    c = np.pad(codes, ((0, 0), (0, codes.shape[1] % 2)))
    return np.ascontiguousarray(c[:, 0::2] | (c[:, 1::2] << 4))


def unpack(packed, K, format):
    if format == "mxfp8":
        return packed
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)[:, :K]


def storage(packed, scales, K, format):
    """Row-major bytes -> the storage order, entry by entry from its description."""
    rows = packed.shape[0]
    per_chunk = 16 if format == "mxfp8" else 32
    step = 3 if format == "mxfp4" else 2      # chunks that a row is filled up to
    per_group = 3 if format == "mxfp4" else 4  # blocks
    chunks = step * -(-K // (step * per_chunk))
    groups = -(-K // (per_group * BLOCK[format]))
    blocks = -(-rows // 128)
    c = np.zeros((blocks, chunks, 128, 16), np.uint8)
    s = np.zeros((blocks, groups, 32, 4, 4), np.uint8)
    for r in range(rows):
        for b in range(packed.shape[1]):
            c[r // 128, b // 16, r % 128, b % 16] = packed[r, b]
        for b in range(scales.shape[1]):
            s[r // 128, b // per_group, r % 32, r % 128 // 32, b % per_group] = scales[r, b]
    return c, s


def random_operand(rng, rows, K, format, exact):
    """(packed, scales, t, 64-bit values).  `exact`: scales near 1, so that sums of some
    thousand products are multiples of 2^-8 below 2^16 and fp32 holds them."""
    block = -(-K // BLOCK[format])
    if format == "mxfp8":
        if exact:  # -8 .. 8 in halves
            q = rng.integers(-16, 17, (rows, K)) / 2.0
            codes = nearest(q, e4m3_values()[:127]) | np.where(q < 0, 128, 0)
        else:
            codes = rng.integers(0, 256, (rows, K))
            codes = np.where(codes & 127 == 127, 0, codes)
    else:
        codes = rng.integers(0, 16, (rows, K))
    codes = codes.astype(np.uint8)
    if format == "nvfp4":
        t = 2.0 ** rng.integers(-11, -7) if not exact else 1.0
        scales = rng.choice([0x30, 0x38, 0x40], (rows, block)) if exact \
            else rng.integers(1, 127, (rows, block))  # 0.5, 1, 2
    else:
        t = 1.0
        scales = 127 + (rng.integers(-1, 2, (rows, block)) if exact
                        else rng.integers(-12, -4, (rows, block)))
    scales = scales.astype(np.uint8)
    return pack(codes, format), scales, float(t), values(codes, scales, format, t)
