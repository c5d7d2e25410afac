"""References and tolerances of the expert-layer tests (numpy, 64 bits).

Tolerance of a sum of n products held in fp32: each of the n additions rounds
or truncates by at most 2^-23 of a partial sum, which is at most S = sum |a b|;
the errors are independent in sign, so they grow like sqrt(n), and 8 covers
short sums: |error| <= (8 + sqrt(n)) * 2^-23 * S.  An fp16 result adds half a
unit in the last place, 2^-11 |result|, and 2^-25 below the normal range.
Small-integer inputs are compared exactly: every product and sum is then a
whole number that fp32 holds.
"""
import numpy as np


def tolerance(ref, abs_sum, n, out):
    tol = (8.0 + np.sqrt(n)) * 2.0 ** -23 * abs_sum
    if out == "f16":
        tol = tol + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    return tol


def assert_within(got, ref, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d off; first at %s: got %r, expected %r"
                             % (what, bad.sum(), bad.size, i, got[i], np.asarray(ref)[i]))


def assert_same(got, ref, out, what=""):
    """Exact: the 64-bit values rounded to the output type."""
    want = np.asarray(ref).astype(np.float16 if out == "f16" else np.float32)
    got = np.asarray(got)
    if not (got == want).all():
        i = tuple(np.argwhere(got != want)[0])
        raise AssertionError("%s: %d of %d differ; first at %s: got %r, expected %r"
                             % (what, (got != want).sum(), got.size, i, got[i], want[i]))


def sort_reference(ids, experts):
    """(offsets, order, position) of the stable sort, dropped slots last."""
    flat = np.asarray(ids).reshape(-1)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(flat.size)
    offsets = np.searchsorted(key[order], np.arange(experts + 1), side="left")
    return offsets, order, position.reshape(np.asarray(ids).shape)


def routing(rng, tokens, topk, experts, drop):
    """Different experts per token, some slots dropped (below 0 or too large)."""
    ids = np.stack([rng.permutation(experts)[:topk] for _ in range(tokens)]) if tokens else \
        np.zeros((0, topk), dtype=np.int64)
    lost = rng.random(ids.shape) < drop
    ids = np.where(lost, rng.choice([-1, -7, experts, 2 ** 31 - 1], ids.shape), ids)
    return ids.astype(np.int32)


def integers(rng, shape, lo=-2, hi=2):
    return rng.integers(lo, hi + 1, shape).astype(np.float16)


def normals(rng, shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float16)


def device(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
