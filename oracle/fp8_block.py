"""Plain numpy forms, in 64 bits, of the block-scaled FP8, expert and block-norm operators: test
infrastructure, written from the definitions in include/apex_w4a4.h and sharing no code with the
CUDA path.  16-bit tensors enter as float64 arrays of their exact values."""
from __future__ import annotations

import numpy as np

MAX = 448.0


def _table():
    """The 127 finite E4M3 magnitudes by code: 4 exponent bits with bias 7, 3 mantissa bits,
    subnormals below 2^-6; code 0x7F is NaN."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    normal = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array((sub + normal)[:127])


TABLE = _table()


def encode(q):
    """E4M3 codes (uint8) of float64 values: nearest, half to even, saturating; NaN -> 0x7F."""
    q = np.asarray(q, dtype=np.float64)
    a = np.minimum(np.abs(q), MAX)
    mids = (TABLE[1:] + TABLE[:-1]) / 2        # exact: table values have few bits
    low = np.searchsorted(mids, a, side="left")    # a tie stays with the lower code
    high = np.searchsorted(mids, a, side="right")
    code = np.where(low % 2 == 0, low, high).astype(np.uint8)
    code = np.where(np.isnan(q), 0x7F, code)
    return (code | np.where(np.signbit(q) & ~np.isnan(q), 0x80, 0)).astype(np.uint8)


def decode(codes):
    t = np.concatenate([TABLE, [np.nan]])
    return np.concatenate([t, -t])[np.asarray(codes, dtype=np.uint8)]


def scale_of(amax):
    """fp32 round-to-nearest of amax / 448 (amax an fp32 value: one IEEE fp32 division)."""
    with np.errstate(all="ignore"):
        return np.asarray(amax, dtype=np.float32) / np.float32(MAX)


def _codes(x, s):
    with np.errstate(all="ignore"):
        q = np.where(s == 0, 0.0, x / s)
    return encode(q)


def quantize_rows(x):
    """x [M, K] -> codes [M, K], scales fp32 [M, ceil(K/128)]."""
    M, K = x.shape
    G = -(-K // 128)
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, G), np.float32)
    for g in range(G):
        part = x[:, 128 * g:128 * g + 128]
        s = scale_of(np.abs(part).max(axis=1))
        scales[:, g] = s
        codes[:, 128 * g:128 * g + 128] = _codes(part, s.astype(np.float64)[:, None])
    return codes, scales


def quantize_blocks(w):
    """w [N, K] -> codes [N, K], scales fp32 [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            scales[i, j] = scale_of(np.abs(w[at]).max())
            codes[at] = _codes(w[at], float(scales[i, j]))
    return codes, scales


def rows_values(codes, scales):
    return decode(codes) * np.repeat(scales.astype(np.float64), 128, axis=1)[:, :codes.shape[1]]


def blocks_values(codes, scales):
    N, K = codes.shape
    full = np.repeat(np.repeat(scales.astype(np.float64), 128, axis=0), 128, axis=1)
    return decode(codes) * full[:N, :K]


def gemm(a_codes, a_scales, w_codes, w_scales):
    """(Y, S): the product, and the sum of its terms' magnitudes, which bounds the rounding."""
    a, w = rows_values(a_codes, a_scales), blocks_values(w_codes, w_scales)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def route(z, k, bias=None, score="softmax", groups=1, topk_groups=1, renormalize=True, scale=1.0,
          mask=None, group_score="top2"):
    """(weights, ids, scores) by a plain loop over the tokens."""
    T, E = z.shape
    weights, ids, scores = np.zeros((T, k)), np.full((T, k), -1, np.int32), np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        row = z[t].astype(np.float64)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                p = 1 / (1 + np.exp(-row))
            elif np.all(row == -np.inf):
                p = np.zeros(E)
            elif np.all(np.isnan(row)):
                p = row
            else:
                p = np.exp(row - np.nanmax(row))
                p = p / p.sum()
        scores[t] = p
        v = p + (0 if bias is None else bias)
        v = np.where(np.isnan(v), -np.inf, v)
        open_ = list(range(E))
        if groups > 1:
            n = E // groups
            if group_score == "top2":
                worth = [sum(sorted(v[g * n:(g + 1) * n])[-2:]) for g in range(groups)]
            else:   # without a bias: by the logits, whose order the scores have
                u = v if bias is not None else np.where(np.isnan(p), -np.inf, row)
                worth = [max(u[g * n:(g + 1) * n]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:topk_groups]
            open_ = [e for e in open_ if e // n in kept]
        if bias is None:      # the order of the scores is that of the logits
            v = np.where(np.isnan(row), -np.inf, row)
        ids[t] = sorted(open_, key=lambda e: (-v[e], e))[:k]
        w = p[ids[t]]
        if renormalize:
            w = w if w.sum() == 0 else w / w.sum()
        weights[t] = w * scale
    return weights, ids, scores


def plan(ids, E):
    flat = np.asarray(ids).ravel()
    lists = [np.flatnonzero(flat == e) for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    order = np.full(flat.size, -1, np.int32)
    order[:offsets[-1]] = np.concatenate(lists)
    return offsets, order


def moe(x, weights, ids, w13_codes, w13_scales, w2_codes, w2_scales):
    """The experts' MLP of x [T, H] float64."""
    E = w13_codes.shape[0]
    xv = rows_values(*quantize_rows(x))
    out = np.zeros_like(xv)
    for e in range(E):
        t, j = np.nonzero(np.asarray(ids) == e)
        if not t.size:
            continue
        g = xv[t] @ blocks_values(w13_codes[e, 0], w13_scales[e, 0]).T
        u = xv[t] @ blocks_values(w13_codes[e, 1], w13_scales[e, 1]).T
        h = rows_values(*quantize_rows(g / (1 + np.exp(-g)) * u))
        y = h @ blocks_values(w2_codes[e], w2_scales[e]).T
        np.add.at(out, t, weights[t, j][:, None] * y)
    return out


def block_norm(x, pre=None, residual=None, post=None, gate=None, alpha=1.0, eps=1e-6, offset=0.0):
    """(h, y), y None without a second norm."""
    def norm(v, w):
        return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * (offset + w)
    z = x if post is None else norm(x, post)
    if gate is not None:
        z = z * np.repeat(gate, x.shape[0] // gate.shape[0], axis=0)
    h = alpha * z + (0 if residual is None else residual)
    return h, None if pre is None else norm(h, pre)
