"""Plain 64-bit (numpy) forms of the layers around the experts, and their tolerances.

u = 2^-24.  Bounds, each from the kernels' own sums and derived before any run:

  rstd        a thread adds up to 32 squares, then 5 shuffles and up to 16 warps: 53
              additions, one rounding in each square's fused step, so the sum is
              within 54 u; division by d and + eps 2 u; halved by the root, 28 u; root
              and reciprocal 2 u: relative 30 u
  norm        two products on top: 32 u relative
  codes       the scale is the largest of values within 32 u, one division: 33 u; what is
              rounded to a code is v (32 u) times 448 / max (33 u), one product: 66 u
  dx          with t = g u (g = dy gamma 1 u, u = s rstd 31 u): mean(t) is within 54 u +
              33 u of mean|t|, one division: 88 u; u mean(t): 31 u + 1; the difference, the
              product with rstd (30 u) and the last sum: 3 u
  dgamma      terms within 31 u; a thread adds `trips` rows, a block 32 lane groups and
              warps at most, the second kernel 19 + 16 partial rows
"""
import numpy as np

import _experts_ref as R

U = R.U


def norm(s, gamma, eps):
    """(v, rstd) of s (fp64)."""
    rstd = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * rstd * gamma, rstd


def norm_tol(v):
    return 32 * U * np.abs(v) + 1e-45


def norm_grad(dy, ds, s, gamma, eps):
    """(dx, its tolerance, dgamma, sum of magnitudes for its tolerance)."""
    rstd = norm(s, gamma, eps)[1]
    unit, g = s * rstd, dy * gamma
    dot, mag = (g * unit).mean(axis=1, keepdims=True), np.abs(g * unit).mean(axis=1, keepdims=True)
    dx = ds + rstd * (g - unit * dot)
    tol = U * rstd * (36 * np.abs(g) + np.abs(unit) * (66 * np.abs(dot) + 88 * mag)) + 2 * U * (np.abs(ds) + np.abs(dx))
    return dx, tol + 1e-44, (dy * unit).sum(axis=0), np.abs(dy * unit).sum(axis=0)


def norm_sums(rows, d):
    """Additions in a sum of dgamma: see above (303 blocks of 256 or 512 threads take rows in turn)."""
    lanes = 8 if d <= 128 else 32
    wpr = 1
    while wpr * 1024 < d:
        wpr *= 2
    per = (512 if wpr > 8 else 256) // (lanes * wpr)
    return -(-rows // (304 * per)) + 32 + 19 + 16 + 31 + 1


def row_codes(v):
    """(block maxima [blocks, rows], v * 448 / max [rows, padded]) of v (fp64)."""
    rows, d = v.shape
    blocks = -(-d // 128)
    p = np.zeros((rows, blocks * 128))
    p[:, :d] = v
    p = p.reshape(rows, blocks, 128)
    m = np.maximum(np.abs(p).max(axis=2), 2.0 ** -100)
    return m.T, (p * (448 / m[:, :, None])).reshape(rows, blocks * 128)


def codes_fit(codes, scale, v):
    """Whether codes (bytes) and scales are those of values within 32 u of v."""
    m, t = row_codes(v)
    if not np.all(np.abs(scale * 448 - m) <= 36 * U * m):
        return False
    got = R.e4m3_values(codes)
    lo, hi = R.e4m3_round(np.clip(t - 66 * U * np.abs(t), -448, 448)), R.e4m3_round(np.clip(t + 66 * U * np.abs(t), -448, 448))
    return bool(np.all((got >= lo) & (got <= hi)))


# ---------------------------------------------------------------------------
# dense layers (torch, fp64)
# ---------------------------------------------------------------------------
# A tensor core's addition may drop, not round, its last bit: within 2 u of the running sum of magnitudes.  bf16: k
# products, 2 k u.  fp32: the first planes' products are read back every 128 of them, 256 u, and added, k / 128 u; the
# five other products are 2^-7 of the magnitudes together and are read back every 4096: 2 * 5 * 2^-7 min(k, 4096) u; what
# is dropped, twice 2^-24, and the planes' own rounding, twice 2^-24: 4 u.  Weight gradients: bf16 too is read back every
# 512 rows; up to 152 parts are added.  The 2-norm of an fp32 result's error: 8 additions that drop 2 u of a running sum,
# which for terms of random sign is no larger than the whole, 16 u.
def sum_bound(dtype, k, mag, gradient=False):
    if dtype == "f32":
        return (256 + k / 128 + 10 / 128 * min(k, 4096) + 4 + (152 if gradient else 0) + 2) * U * mag
    return (2 * (min(k, 512) if gradient else k) + (k / 512 + 152 if gradient else 0) + 2) * U * mag


def act64(act, z):
    import torch
    s = torch.sigmoid(z)
    phi = 0.5 * (1 + torch.erf(z / 2 ** 0.5))
    return {"none": (z, torch.ones_like(z)), "relu": (z.clamp(min=0), (z > 0).to(z.dtype)),
            "sigmoid": (s, s * (1 - s)), "silu": (z * s, s * (1 + z * (1 - s))),
            "gelu": (z * phi, phi + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5)}[act]


def act_tol(z, y, tol_z):
    """Of act(z) with z within tol_z: slopes are at most 1.13; expf and erff are within 2 ulp, then a sum, a division
    and a product: 10 u (|z| + 1)."""
    return 1.13 * tol_z + 10 * U * (z.abs() + 1) + U * y.abs()


def fits(got, ref, tol, dtype):
    """R.within for torch tensors."""
    import torch
    if dtype == "f32":
        return bool(((got.double() - ref).abs() <= tol).all())
    lo, hi = (ref - tol).to(torch.bfloat16), (ref + tol).to(torch.bfloat16)
    return bool(((got >= lo) & (got <= hi)).all())


def dz64(dtype, act, dy, pre):
    """(dz as the products have it, how far it may be off): rounded to bf16 where the inputs are bf16."""
    import torch
    dz = dy * act64(act, pre)[1]
    err = 16 * U * (1 + pre.abs()) * dy.abs() if act != "none" else 0 * dy
    if dtype == "f32":
        return dz, err, dz, err
    mid = dz.to(torch.bfloat16).double()
    lo, hi = (dz - err).to(torch.bfloat16).double(), (dz + err).to(torch.bfloat16).double()
    return mid, torch.maximum(hi - mid, mid - lo), dz, err


# ---------------------------------------------------------------------------
# balanced routing
# ---------------------------------------------------------------------------
def balanced(s, k, score, bias, groups, group_k, renorm, factor):
    """(expert, weight, slot, token, offsets, p) of scores s (fp64)."""
    s = np.array(s, dtype=np.float64)
    T, E = s.shape
    s[(np.isnan(s) | (s == np.inf)).any(axis=1)] = -np.inf
    b = np.zeros(E) if bias is None else np.where(np.asarray(bias) < np.inf, np.asarray(bias, dtype=np.float64), -np.inf)
    live = s > -np.inf
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            p = np.where(live, 1 / (1 + np.exp(-s)), 0.0)
        else:
            m = np.where(live.any(axis=1), s.max(axis=1, initial=-np.inf), 0.0)[:, None]
            p = np.where(live, np.exp(s - m), 0.0)
            p = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
    key = np.where(live, p + b, -np.inf)
    if group_k < groups:
        per = E // groups
        member = -np.sort(-key.reshape(T, groups, per), axis=2)[:, :, :2]
        worth = np.where(np.isfinite(member), member, 0.0).sum(axis=2)
        worth = np.where(np.isfinite(member).any(axis=2), worth, -np.inf)
        stay = np.argsort(-worth, axis=1, kind="stable")[:, :group_k]
        kept = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(kept, stay, True, axis=1)
        key = np.where(np.repeat(kept, per, axis=1), key, -np.inf)
    # without a bias the scores' order is the keys'
    order = np.argsort(-(key if bias is not None else np.where(key > -np.inf, s, -np.inf)), axis=1, kind="stable")[:, :k]
    has = np.take_along_axis(key, order, 1) > -np.inf
    w = np.where(has, np.take_along_axis(p, order, 1), 0.0)
    if renorm:
        if score == "sigmoid":   # in proportion, whatever 64 bits can hold
            ls = np.where(has, -np.logaddexp(0, -np.take_along_axis(s, order, 1)), -np.inf)
            w = np.where(has, np.exp(ls - np.where(has.any(axis=1), ls.max(axis=1), 0.0)[:, None]), 0.0)
        w = w / np.where(w.sum(axis=1) > 0, w.sum(axis=1), 1.0)[:, None]
    expert = np.where(has, order, -1).astype(np.int32)
    flat = np.where(has, order, E).ravel()
    at = np.argsort(flat, kind="stable")
    count = int(has.sum())
    slot, token = np.full(T * k, -1, dtype=np.int32), np.full(T * k, -1, dtype=np.int32)
    slot[at[:count]] = np.arange(count)
    token[:count] = at[:count] // k
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]).astype(np.int32)
    return expert, factor * w, slot.reshape(T, k), token, offsets, p


def balanced_grad(dw, s, score, renorm, factor, expert, p):
    """(dscores, magnitudes that its tolerance goes by) for choices `expert` and score functions p."""
    T, E = s.shape
    has = expert >= 0
    at = np.where(has, expert, 0)
    pj = np.where(has, np.take_along_axis(p, at, 1), 0.0)
    if renorm:
        sj = np.take_along_axis(s, at, 1)
        ls = np.where(has, -np.logaddexp(0, -sj) if score == "sigmoid" else sj, -np.inf)
        wj = np.where(has, np.exp(ls - np.where(has.any(axis=1), ls.max(axis=1), 0.0)[:, None]), 0.0)
        wj = wj / np.where(wj.sum(axis=1) > 0, wj.sum(axis=1), 1.0)[:, None]
    else:
        wj = pj
    g = np.where(has, factor * dw, 0.0)
    dot, mag = (wj * g).sum(axis=1, keepdims=True), np.abs(wj * g).sum(axis=1, keepdims=True)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    if score == "softmax" and not renorm:
        full = np.zeros((T, E))
        t, j = np.nonzero(has)
        full[t, expert[t, j]] = g[t, j]
        routed = has.any(axis=1, keepdims=True)
        return np.where(routed, p * (full - dot), 0.0), np.abs(p * full) + p * mag
    slope = 1 - pj if score == "sigmoid" else np.ones_like(pj)
    d = wj * (g - dot) * slope if renorm else wj * g * slope
    m = (np.abs(wj * g) + (wj * mag if renorm else 0)) * (slope if score == "softmax" else 1)
    t, j = np.nonzero(has)
    out[t, expert[t, j]], size[t, expert[t, j]] = d[t, j], m[t, j]
    return out, size
