"""Plain 64-bit (numpy) forms of the expert layer's operators, and its tolerances.

u = 2^-24 is fp32's unit roundoff.  A result that is rounded to bf16 at the end
has to lie between the roundings of its fp32 bound's two ends (rounding keeps
order), which leaves no slack of its own.  Bounds used by the tests (each derived from the kernels' own
sums, before any run):

  softmax weight   expf is within 2 ulp, the sum has at most E terms, one division:
                   relative (E + 8) u
  score gradient   p (g - sum p g): (2E + 24) u (|p g| + |p| sum |p g|)
  weighted rows    k fused multiply-adds: k u sum |w r|
  weight gradient  d fused multiply-adds in any order: d u sum |dy r|
  e4m3 product     a block's 128 products are exact in fp32 and added by the tensor
                   cores; an addition may drop, not round, its last bit, so each is
                   within 2 u of the running sum of magnitudes: 256 u per block;
                   scaling and adding kb blocks: (kb + 3) u; together
                   (256 + kb + 3) u sum |a b|
  norm             partial sums of at most 8 x 8192 / 256 = 256 squares an
                   accumulator in fp32, two joins, then fp64: relative 129 u in the
                   root (half of 258), and one rounding
"""
import numpy as np
import torch

U = 2.0 ** -24


def within(got, ref, tol, dtype):
    """Whether every result is one that an fp32 value within tol of ref can be stored as in dtype."""
    got = np.asarray(got, dtype=np.float64)
    if dtype == "f32":
        return bool(np.all(np.abs(got - ref) <= tol))
    lo, hi = (torch.from_numpy(np.asarray(v)).to(torch.bfloat16).double().numpy() for v in (ref - tol, ref + tol))
    return bool(np.all((got >= lo) & (got <= hi)))


def route(s, k, renorm):
    """(expert, weight, slot, token, offsets, p) of scores s (fp64); p is the softmax the weights come from."""
    s = np.asarray(s, dtype=np.float64)
    T, E = s.shape
    bad = (np.isnan(s) | (s == np.inf)).any(axis=1)
    s = np.where(bad[:, None], -np.inf, s)
    order = np.argsort(-s, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(s, order, 1)
    live = top > -np.inf
    m = np.where(live[:, :1], top[:, :1], 0.0)
    z = np.where(s > -np.inf, np.exp(s - m), 0.0)
    if renorm:
        keep = np.zeros((T, E), dtype=bool)
        keep[np.arange(T)[:, None], order] = live
        z = z * keep
    total = z.sum(axis=1, keepdims=True)
    p = z / np.where(total > 0, total, 1.0)
    weight = np.where(live, np.take_along_axis(p, order, 1), 0.0)
    expert = np.where(live, order, -1).astype(np.int32)
    slot = np.full((T, k), -1, dtype=np.int32)
    token = np.full(T * k, -1, dtype=np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    r = 0
    for e in range(E):
        t, j = np.nonzero(expert == e)           # by token: a token chooses an expert once
        slot[t, j] = r + np.arange(t.size)
        token[r:r + t.size] = t
        r += t.size
        offsets[e + 1] = r
    return expert, weight, slot, token, offsets, p


def route_grad(dw, s, k, renorm):
    expert, _, _, _, _, p = route(s, k, renorm)
    g = np.zeros_like(p)
    t, j = np.nonzero(expert >= 0)
    g[t, expert[t, j]] = dw[t, j]
    dot = (p * g).sum(axis=1, keepdims=True)
    mag = np.abs(p * g) + np.abs(p) * np.abs(p * g).sum(axis=1, keepdims=True)
    return p * (g - dot), mag


def e4m3_round(v):
    """Values of the e4m3 codes nearest to fp32 values v (ties to even, saturating)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 448.0)
    with np.errstate(divide="ignore"):
        ex = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (ex - 3)
    return np.sign(v) * np.rint(a / step) * step


def e4m3_values(codes):
    """Values of e4m3 code bytes."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex.astype(np.float64) - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def scale_of(amax):
    """(scale, multiplier) of a block's largest magnitude, in fp32 as defined."""
    m = np.maximum(np.asarray(amax, dtype=np.float32), np.float32(2.0 ** -100))
    return (m / np.float32(448)).astype(np.float32), (np.float32(448) / m).astype(np.float32)


def quantize(x, rows_per_scale, cols_per_scale):
    """Code values [R, C] (fp64) and scales [ceil(R / r), ceil(C / c)] of x (fp32 values), one scale per block."""
    x = np.asarray(x, dtype=np.float32)
    R, C = x.shape
    r, c = rows_per_scale, cols_per_scale
    nr, nc = -(-R // r), -(-C // c)
    p = np.zeros((nr * r, nc * c), dtype=np.float32)
    p[:R, :C] = x
    p = p.reshape(nr, r, nc, c)
    s, inv = scale_of(np.abs(p).max(axis=(1, 3)))
    q = e4m3_round(p * inv[:, None, :, None])
    return q.reshape(nr * r, nc * c)[:R, :C], s


def spread(s, r, c, R, C):
    """A block scale for every element."""
    return np.repeat(np.repeat(s.astype(np.float64), r, 0)[:R], c, 1)[:, :C]


def product_bound(mag, kb):
    return (256 + kb + 3) * U * mag
