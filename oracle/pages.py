"""fp64 references of page-sparse decoding and 4-bit weights (test infrastructure only).

Written from the definitions with plain numpy; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def page_keys(rows, P):
    """Means of the pages of rows [S][D], and of their magnitudes: [pages][D] each."""
    S = rows.shape[0]
    cut = [rows[i: i + P].astype(np.float64) for i in range(0, S, P)]
    return np.stack([c.mean(0) for c in cut]), np.stack([np.abs(c).mean(0) for c in cut])


def page_scores(q_lat, keys, see, P, scale):
    """Scores [pages] of one query token q_lat [H][D] that sees `see` tokens, on page keys [pages][D];
    the heads' normalisers [H] and the largest score magnitude scale * sum_d |q_d k_d|."""
    n = -(-see // P)
    k = keys[:n].astype(np.float64)
    count = np.minimum(P, see - P * np.arange(n)).astype(np.float64)
    z = scale * (q_lat.astype(np.float64) @ k.T)
    mag = scale * (np.abs(q_lat).astype(np.float64) @ np.abs(k).T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top) * count
    total = e.sum(1, keepdims=True)
    return (e / total).sum(0), (top + np.log(total))[:, 0], mag.max()


def select_pages(scores, n, budget, sinks, recent):
    """The list [budget] of a query that sees n pages."""
    if n <= budget:
        keep = np.arange(n)
    else:
        mid = np.arange(sinks, n - recent)
        s = np.asarray(scores[sinks: n - recent], np.float64)
        nan = np.isnan(s)
        order = np.lexsort((mid, -np.where(nan, 0.0, s), nan))
        best = np.sort(mid[order[: budget - sinks - recent]])
        keep = np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)])
    out = np.full(budget, -1, np.int32)
    out[: len(keep)] = keep
    return out


def attend_pages(q_lat, rows, pages, see, P, d_c, scale):
    """Output [H][d_c] and LSE [H] of one query token over the tokens below `see` of its pages; the
    largest score magnitude and sum_j p_j |c_j| [H][d_c]."""
    H = q_lat.shape[0]
    at = np.concatenate([np.arange(p * P, min(see, p * P + P)) for p in pages if p >= 0] or [np.zeros(0, int)])
    if at.size == 0:
        return np.zeros((H, d_c)), np.full(H, -np.inf), 0.0, np.zeros((H, d_c))
    x = rows[at].astype(np.float64)
    z = scale * (q_lat.astype(np.float64) @ x.T)
    mag = scale * (np.abs(q_lat).astype(np.float64) @ np.abs(x).T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    return p @ x[:, :d_c], (top + np.log(total))[:, 0], mag.max(), p @ np.abs(x[:, :d_c])


def mx4_quantize(W):
    """Codes [K][N] (bit 3 the sign) and exponents [K / 32][N] of W."""
    W = np.asarray(W, np.float64)
    K, N = W.shape
    b = W.reshape(K // 32, 32, N)
    top = np.abs(b).max(1)
    frac, ex = np.frexp(top)                       # top = frac 2^ex, frac in [1/2, 1)
    e = np.where(top > 0, ex - 1 + (frac >= 0.875) - 2, -127)
    e = np.clip(e, -127, 125)
    y = np.abs(b) / np.exp2(e.astype(np.float64))[:, None]
    d = np.abs(y[..., None] - GRID)                # nearest, half-way values to the even code
    near = d.min(-1, keepdims=True)
    tie = d == near
    even = tie & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))
    code = np.where(y > 6.0, 7, code) | (np.signbit(b) << 3)
    return code.reshape(K, N).astype(np.uint8), e


def mx4_values(code, e):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(e.shape[0], 32, -1) * np.exp2(e.astype(np.float64))[:, None]).reshape(code.shape)


def mx4_pack(code, e):
    """The arrays as the library lays them out: codes [N][K / 2], scales [tiles][groups][32][4][4]."""
    K, N = code.shape
    c = np.ascontiguousarray(code.T)
    packed = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    scales = np.full((-(-N // 128), -(-K // 128), 32, 4, 4), 127, np.uint8)
    for n in range(N):
        for kb in range(K // 32):
            scales[n // 128, kb // 4, n % 32, (n % 128) // 32, kb % 4] = e[kb, n] + 127
    return packed, scales
