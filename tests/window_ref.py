"""Plain 64-bit attention of rows at positions, under a window with first tokens that stay visible, for the tests."""
import numpy as np


def sees(pos, T, window, sinks):
    """[rows][T]: whether the row at pos[r] sees token t."""
    t, p = np.arange(T)[None], np.asarray(pos)[:, None]
    see = t <= p
    return see & ((t > p - window) | (t < sinks)) if window else see


def rows(q, k, v, pos, scale, window=0, sinks=0):
    """Rows q [R][Hq][D] at pos over k, v [T][Hk][D] (float64): out, lse, sum p |v|, and the largest of scale sum |q k| over
    the keys that a row sees (what the rounding of K moves a score by, per unit)."""
    R, Hq, D = q.shape
    T, Hk = k.shape[:2]
    out, mag = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    lse, most = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
    see = sees(pos, T, window, sinks)
    some = see.any(1)
    if T == 0 or not some.any():
        return out, lse, mag, most
    for h in range(Hq):
        g = h * Hk // Hq
        with np.errstate(invalid="ignore"):
            s = np.where(see, scale * (q[:, h] @ k[:, g].T), -np.inf)[some]
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            lse[some, h] = m[:, 0] + np.log(p.sum(1))
            p /= p.sum(1, keepdims=True)
            out[some, h], mag[some, h] = p @ v[:, g], p @ np.abs(v[:, g])
            most[:, h] = np.where(see, abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, g]).T), 0).max(1)
    return out, lse, mag, most
