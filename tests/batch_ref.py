"""Plain 64-bit forms of the batch operators (kvs_prompt_*, kvs_q4_*) for the tests: numpy, one row at a time."""
import math

import numpy as np


def q4_encode(x):
    """Q4_0 of the last axis (fp32 steps): codes 0..15 and fp16 scales per 32-block."""
    blk = np.ascontiguousarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, 32)
    at = np.abs(blk).argmax(-1)[..., None]
    d = np.take_along_axis(blk, at, -1)[..., 0] / np.float32(-8)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(d != 0, np.float32(1) / np.where(d != 0, d, np.float32(1)), np.float32(0)).astype(np.float32)
        y = (blk * inv[..., None]).astype(np.float32) + np.float32(8.5)
    codes = np.clip(np.trunc(np.nan_to_num(y, nan=0.0)), 0, 15).astype(np.uint8)
    return codes, d.astype(np.float16)


def q4_values(codes, scales):
    """float64 [..., D] of codes [..., NB, 32] and scales [..., NB]."""
    v = (codes.astype(np.float64) - 8) * scales.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


def q4_tile(kcodes, kscales, vcodes, vscales):
    """One 36 D byte tile from codes [32][NB][32] and scales [32][NB], by the formulas include/kvs.h states."""
    NB = kscales.shape[1]
    D = NB * 32
    out = np.zeros(36 * D, np.uint8)
    half = out.view(np.float16)
    for t in range(32):
        for b in range(NB):
            for j in range(16):
                u = t // 8 * NB + b
                out[((u // 4 * 32) + t % 8 * 4 + j // 4) * 16 + u % 4 * 4 + j % 4] = kcodes[t, b, j] | kcodes[t, b, j + 16] << 4
                w = (t // 16 * NB + b) * 2 + t % 4 // 2
                out[18 * D + ((w // 4 * 32) + j % 8 * 4 + t % 16 // 4) * 16 + w % 4 * 4 + t % 2 * 2 + j // 8] = \
                    vcodes[t, b, j] | vcodes[t, b, j + 16] << 4
            half[8 * D + ((t // 16 * 8 + t % 8) * NB + b) * 2 + t // 8 % 2] = kscales[t, b]
            half[17 * D + (t // 4 * NB + b) * 4 + t % 4] = vscales[t, b]
    return out


def prompt(q, k, v, scale):
    """One prompt, float64 [L][H][D]: out, lse and sum_j p_ij |v_j| (the scale of the rounding errors)."""
    L, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse, mag = np.zeros((L, Hq, D)), np.zeros((L, Hq)), np.zeros((L, Hq, D))
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h // G].T)
        s[np.triu_indices(L, 1)] = -np.inf
        m = s.max(1)
        p = np.exp(s - m[:, None])
        lse[:, h] = m + np.log(p.sum(1))
        p /= p.sum(1, keepdims=True)
        out[:, h], mag[:, h] = p @ v[:, h // G], p @ np.abs(v[:, h // G])
    return out, lse, mag


def prompt_weights(q, k, lse, scale, window=0):
    """One prompt's [Hk][L] weights under the given lse."""
    L, Hq, _ = q.shape
    Hk = k.shape[1]
    r0 = max(0, L - window) if window else 0
    w = np.zeros((Hk, L))
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h * Hk // Hq].T)
        p = np.exp(s - lse[:, h, None])
        p[np.triu_indices(L, 1)] = 0
        w[h * Hk // Hq] += p[r0:].sum(0)
    return w


def attend(q, k, v, scale):
    """Rows q [R][Hq][D] over k, v [T][Hk][D]; row r sees T - R + r + 1 tokens: out, lse, sum p |v|."""
    R, Hq, D = q.shape
    T, Hk = k.shape[:2]
    out, lse, mag = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf), np.zeros((R, Hq, D))
    for r in range(R):
        n = max(0, T - R + r + 1)
        if n == 0:
            continue
        for h in range(Hq):
            s = scale * (k[:n, h * Hk // Hq] @ q[r, h])
            m = s.max()
            p = np.exp(s - m)
            lse[r, h] = m + math.log(p.sum())
            p /= p.sum()
            out[r, h], mag[r, h] = p @ v[:n, h * Hk // Hq], p @ np.abs(v[:n, h * Hk // Hq])
    return out, lse, mag


def cache_weights(q, k, lse, scale):
    """[Hk][T] weights of rows q under the given lse [R][Hq]."""
    R, Hq, _ = q.shape
    T, Hk = k.shape[:2]
    w = np.zeros((Hk, T))
    for r in range(R):
        n = max(0, T - R + r + 1)
        for h in range(Hq):
            if n:
                w[h * Hk // Hq, :n] += np.exp(scale * (k[:n, h * Hk // Hq] @ q[r, h]) - lse[r, h])
    return w


def evict(weights, keep, sinks, recent):
    """Kept token indices of one [T] weight row."""
    T = len(weights)
    if T <= keep:
        return np.arange(T)
    mid = np.arange(sinks, T - recent)
    w = weights[mid].astype(np.float64)
    rank = np.where(np.isnan(w), 0, 1)
    order = np.lexsort((mid, -np.where(np.isnan(w), 0, w), -rank))
    chosen = mid[order[:keep - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), chosen, np.arange(T - recent, T)]))
