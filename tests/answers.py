"""Plain 64-bit forms of the operators between a hidden state and text, on the
host, written from the formulas, and the tolerances their tests use."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128
TINY = 2.0 ** -126


def half_step(dtype) -> float:
    """Largest error of rounding to dtype, relative to the value."""
    return torch.finfo(dtype).eps / 2


def spread(scales, n, k, rows_too):
    """Scales of blocks as an array of the whole matrix's shape."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)[:, :k]
    return np.repeat(s, BLOCK, axis=0)[:n] if rows_too else s


def norm(x, residual, weight, eps):
    """(y, h) in 64 bits: the normed rows before they are put into 8 bits."""
    h = x.double().cpu().numpy()
    if residual is not None:
        h = h + residual.double().cpu().numpy()
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight.double().cpu().numpy()
    return y, h


def block_max(y, rows_too=False):
    """Largest magnitude of each block of 128 columns (and 128 rows)."""
    a = np.abs(y)
    at = np.arange(0, y.shape[1], BLOCK)
    a = np.maximum.reduceat(a, at, axis=1)
    if rows_too:
        a = np.maximum.reduceat(a, np.arange(0, y.shape[0], BLOCK), axis=0)
    return a


def product(a, sa, b, sb):
    """(a b^T with scales in 64 bits, the same with every term's magnitude)."""
    m, k = a.shape
    n = b.shape[0]
    fa = a.float().cpu().numpy().astype(np.float64) * spread(sa.cpu().numpy(), m, k, False)
    fb = b.float().cpu().numpy().astype(np.float64) * spread(sb.cpu().numpy(), n, k, True)
    return fa @ fb.T, np.abs(fa) @ np.abs(fb).T


def product_tolerance(magnitude, blocks):
    """A block's 128 exact products are added in f32 in some order, at worst
    by truncation: 128 * 2^-23 of the magnitudes' sum. The factor of two
    scales, its product and the sum over blocks round to nearest."""
    return magnitude * (128 * 2.0 ** -23 + (blocks + 3) * 2.0 ** -24)


def product_dropped(a, sa, b, sb):
    """What the e4m3 matrix instructions may drop: of 8 neighbouring products
    all but the largest lose up to 2^-13 of its power of two."""
    m, k = a.shape
    n = b.shape[0]
    fa = np.abs(a.float().cpu().numpy().astype(np.float64) * spread(sa.cpu().numpy(), m, k, False))
    fb = np.abs(b.float().cpu().numpy().astype(np.float64) * spread(sb.cpu().numpy(), n, k, True))
    out = np.zeros((m, n))
    for at in range(0, k, 8):
        best = np.zeros((m, n))
        for c in range(at, min(k, at + 8)):
            np.maximum(best, fa[:, c, None] * fb[None, :, c], out=best)
        out += 7 * 2.0 ** -13 * best
    return out


# Products that between them take every kernel there is (see
# test_answer_plan.py, which asks the library's own rule), each with what rows
# of a cover: (m, n, k).
PRODUCTS = [
    # streams over parts of K: 16, 32 and 64 rows of a
    (2, 1700, 2048), (30, 3300, 2049), (61, 4256, 2064), (130, 456, 2064), (600, 456, 2049),
    # streams: up to 16, 32 and 64 rows
    (1, 20000, 400), (9, 700, 100), (30, 1000, 272), (60, 700, 513),
    # 128 x 64 tiles: whole, short and odd rows, and rows of less than a block
    (5, 6200, 256), (64, 6200, 400), (33, 16100, 401), (64, 12500, 100),
    # 256 x 256, with few and with many blocks of K
    (520, 16640, 384), (500, 32700, 2048),
    # 256 x 128: whole and short rows
    (600, 8256, 1024), (515, 8000, 528), (600, 16500, 272),
    # 128 x 128 by four waves: whole, short and odd rows, and rows of less than a block
    (789, 9244, 128), (789, 9244, 144), (200, 1000, 512), (200, 1000, 528), (515, 9000, 529), (300, 700, 100),
    # by eight waves (exact sums): whole, short and odd rows
    (128, 12500, 256), (128, 12500, 272), (128, 12500, 257),
]


def draw(row, u, temperature, top_k, top_p, min_p):
    """(id, log of its share) for one row of logits, by the definition: NaN
    never kept, +inf the largest finite f32."""
    x = np.asarray(row, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    if not (x > -np.inf).any():
        return -1, -math.inf
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if not temperature > 0 or top_p <= 0:
        return int(order[0]), 0.0
    w = np.exp((x[order] - x[order[0]]) / temperature)
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        run = np.cumsum(w)
        stop = int(np.argmax(run >= top_p * run[-1])) + 1
        order, w = order[:stop], w[:stop]
    if min_p > 0:
        order, w = order[w >= min(min_p, 1.0)], w[w >= min(min_p, 1.0)]
    ids = np.sort(order)
    t = (x[ids] - x[order[0]]) / temperature
    run = np.cumsum(np.exp(t))
    if not u > 0:
        at = 0
    else:
        hit = run > min(u, 1 - 2.0 ** -24) * run[-1] if u < 1 else run >= run[-1]
        at = int(np.argmax(hit))
    return int(ids[at]), float(t[at] - math.log(run[-1]))


def strings(merges):
    text = [bytes([i]) for i in range(256)]
    for left, right in np.asarray(merges).reshape(len(merges), -1)[:, :2].tolist():
        text.append(text[left] + text[right])
    return text


def merge_list(n, seed, longest=24):
    """A list of n merges whose strings have up to `longest` bytes."""
    r = np.random.RandomState(seed)
    size = [1] * 256
    merges = []
    for k in range(n):
        left, right = int(r.randint(256 + k)), int(r.randint(256 + k))
        if size[left] + size[right] > longest:
            left, right = int(r.randint(256)), int(r.randint(256))
        merges.append((left, right, n - k))
        size.append(size[left] + size[right])
    return np.array(merges, dtype=np.int32).reshape(n, 3)
