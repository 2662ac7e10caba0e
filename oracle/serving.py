"""fp64 references of the shared-prefix and eviction calls (test infrastructure only).

Written from the definitions with plain numpy; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .mla import e4m3_encode, e4m3_decode, rope


def expand_prefix(c, W_UK, W_UV, H):
    """keys [H][L][d_n] and values [H][L][d_v] of latents c [L][d_c]; with the sums of the
    products' magnitudes (for error bounds)."""
    c = np.asarray(c, np.float64)

    def heads(W):
        W = np.asarray(W, np.float64)
        x = c @ W
        mag = np.abs(c) @ np.abs(W)
        return tuple(np.stack(np.split(y, H, axis=1)) for y in (x, mag))

    (K, aK), (V, aV) = heads(W_UK), heads(W_UV)
    return K, V, aK, aV


def attend_prefix(q_nope, q_pe, keys, values, k_pe, seq_lens, scale, theta=10000.0):
    """u [B][q][H][d_v], lse [B][q][H], and for error bounds: the largest score magnitude sum
    max_l scale * sum_d |q_d k_d| [B][q][H] and sum_l p_l |v_l| [B][q][H][d_v]."""
    B, q, H, _ = q_nope.shape
    L = k_pe.shape[0]
    u = np.zeros((B, q, H, values.shape[2]))
    mag_v = np.zeros_like(u)
    lse = np.full((B, q, H), -np.inf)
    mag_s = np.zeros((B, q, H))
    keys, values, k_pe = (np.asarray(x, np.float64) for x in (keys, values, k_pe))
    for b in range(B):
        S = int(seq_lens[b])
        if S < q or L == 0:
            continue
        for t in range(q):
            pos = L + S - q + t
            qn = np.asarray(q_nope[b, t], np.float64)
            qr = rope(np.asarray(q_pe[b, t], np.float64), np.full(H, pos), theta)
            s = scale * (np.einsum("hd,hld->hl", qn, keys) + qr @ k_pe.T)
            mag = scale * (np.einsum("hd,hld->hl", np.abs(qn), np.abs(keys)) + np.abs(qr) @ np.abs(k_pe).T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(1, keepdims=True)
            u[b, t] = np.einsum("hl,hlv->hv", e / l, values)
            mag_v[b, t] = np.einsum("hl,hlv->hv", e / l, np.abs(values))
            lse[b, t] = (m + np.log(l))[:, 0]
            mag_s[b, t] = mag.max(1)
    return u, lse, mag_s, mag_v


def join_prefix(o_lat, lse, u_prefix, lse_prefix, W_UV, H):
    """u [R][H][d_v]: the own tokens' lifted output and the prefix's under their softmax weights."""
    R = o_lat.shape[0]
    own = np.einsum("rhc,chv->rhv", o_lat.reshape(R, H, -1).astype(np.float64),
                    np.asarray(W_UV, np.float64).reshape(W_UV.shape[0], H, -1))
    top = np.maximum(lse, lse_prefix)
    safe = np.where(np.isneginf(top), 0.0, top)
    ea, eb = np.exp(lse - safe), np.exp(lse_prefix - safe)
    tot = np.where(ea + eb > 0, ea + eb, 1.0)
    a, b = (ea / tot)[..., None], (eb / tot)[..., None]
    up = u_prefix.reshape(R, H, -1)
    return np.where(a > 0, a * own, 0.0) + np.where(b > 0, b * up, 0.0)


def key_weights(q_lat, lse, rows, old, q_len, scale, decay):
    """weights [S] of one request: q_lat [q][H][D], lse [q][H], rows [S][D], old [>= S]; and the
    bound scale * sum_d |q_d x_d| of the scores, [S] (the largest over heads and tokens)."""
    S = rows.shape[0]
    mass, mag = np.zeros(S), np.zeros(S)
    for t in range(q_len):
        n = S - q_len + t + 1
        z = scale * (rows[:n] @ q_lat[t].T.astype(np.float64))
        a = scale * (np.abs(rows[:n]) @ np.abs(q_lat[t]).T.astype(np.float64))
        mass[:n] += np.exp(z - lse[t][None]).sum(1)
        mag[:n] = np.maximum(mag[:n], a.max(1))
    out = mass.copy()
    if decay:
        out[: S - q_len] += decay * old[: S - q_len].astype(np.float64)
    return out, mag


def evict_order(weights, S, budget, sinks, recent):
    """Ascending indices that an eviction of S tokens to `budget` keeps."""
    if S <= budget:
        return np.arange(S)
    mid = np.arange(sinks, S - recent)
    w = np.asarray(weights[sinks: S - recent], np.float64)
    nan = np.isnan(w)
    # NaN behind every number, -inf included; equal weights by index
    order = np.lexsort((mid, -np.where(nan, 0.0, w), nan))
    best = np.sort(mid[order[: budget - sinks - recent]])
    return np.concatenate([np.arange(sinks), best, np.arange(S - recent, S)])


def turn_rows(k, delta, theta=10000.0):
    """Rotary keys k [n][d_r] turned by delta [n] positions."""
    return rope(np.asarray(k, np.float64), np.asarray(delta), theta)


def turn_codes(codes, delta, theta=10000.0):
    """The same on e4m3 codes: (turned values, nearest codes)."""
    y = turn_rows(e4m3_decode(codes), delta, theta)
    return y, e4m3_encode(y)
