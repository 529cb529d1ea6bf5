"""Plain 64-bit references of the operators around the experts (numpy), and the
bounds their GPU results are held to.

Bounds are counted in roundings: rounding to a type is off by at most half a
step, relative eps / 2 (bf16 2^-8, fp16 2^-11, fp32 2^-24), or half the smallest
subnormal; a sum of n products in fp32, in any order, is off by at most
n * 2^-24 (1 + small) times the sum of the products' magnitudes (each product
enters at most n roundings, its own among them)."""
import numpy as np
import torch

U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def f64(t):
    return t.detach().cpu().double().numpy()


def stored(bound, y, dtype):
    """The error bound of a value y that was computed within `bound` and then
    rounded to dtype."""
    return bound + (np.abs(y) + bound) * HALF[dtype] + TINY[dtype]


def sort_routes(ids, E):
    flat = np.asarray(ids, np.int64).reshape(-1)
    here = (flat >= 0) & (flat < E)
    perm = np.argsort(np.where(here, flat, E), kind="stable")
    kept = int(here.sum())
    row_to_route = np.where(np.arange(flat.size) < kept, perm, -1)
    route_to_row = np.full(flat.size, -1, np.int64)
    route_to_row[perm[:kept]] = np.arange(kept)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[here], minlength=E))])
    return row_to_route, route_to_row, offsets


def quantize(x):
    """(codes, scales) of a float64 matrix whose values are representable in fp32."""
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axis=1)
        s = (top / 127.0).astype(np.float32).astype(np.float64)
        ok = np.isfinite(s) & (s > 0)
        q = np.rint(x / np.where(ok, s, 1.0)[:, None])
        codes = np.where(ok[:, None], np.clip(q, -127, 127), 0.0)
    return codes.astype(np.int8), s


def matmul(a, sa, b, sb, bias=None):
    """(y, bound): the product in 64 bits, and how far its fp32 scaling may be off
    before the result is rounded: the sum to fp32, times sa, then the fma with sb
    (and bias), each one rounding of a value near the scaled sum."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T
    y = acc * sa[:, None] * sb[None, :]
    bound = 3.01 * U32 * np.abs(y)
    if bias is not None:
        y = y + bias[None, :]
        bound = bound + U32 * np.abs(y)
    return y, bound


def assert_within(got, want, bound, what):
    got = f64(got)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err - bound):.3e} over its bound"
