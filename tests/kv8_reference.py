"""Plain 64-bit forms of the 8-bit cache and of the log probabilities (numpy, CPU), written from their formulas.

Bounds.  A code of e4m3 is off by at most 2^-4 of the value it stands for where it is normal, and by half of the least
step, 2^-10, of the vector's power of two below 2^-6 of it.  A rotated value is computed in fp32: two products and a sum,
each rounded to 2^-24 of itself."""
import numpy as np

E4M3 = 2.0 ** -4


def e4m3_values():
    """The value of each of the 256 codes; NaN for 0x7f and 0xff."""
    b = np.arange(256)
    sign, e, m = np.where(b & 128, -1.0, 1.0), b >> 3 & 15, b & 7
    val = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.astype(float) - 7))
    return sign * np.where((b & 127) == 127, np.nan, val)


VALUES = e4m3_values()


def exponent_byte(x):
    """Of vectors x [.., D] in 64 bits: the smallest power of two under which all are at most 448, at least 2^-126."""
    top = np.abs(x).max(-1)
    with np.errstate(invalid="ignore"):
        e = np.array([-126 if not (t > 0 and np.isfinite(t)) else next(
            k for k in range(max(-126, int(np.floor(np.log2(t))) - 10), 200) if t <= 448 * 2.0 ** k) for t in top.ravel()])
    e = np.maximum(e.reshape(top.shape), -126)
    return np.where(np.isfinite(top), e + 127, 255).astype(np.uint8)


def codes(x, byte):
    """The nearest codes of x [.., D] under exponent bytes [..], ties to the even code."""
    y = np.where(byte[..., None] == 255, 0.0, x * 2.0 ** (127.0 - byte[..., None]))
    grid = VALUES[:127]  # 0 .. 448, ascending with the code
    a = np.abs(y)
    i = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    code = np.where(up, i, i - 1)
    return np.where(np.signbit(y), code | 128, code).astype(np.uint8)


def values(code, byte):
    with np.errstate(invalid="ignore"):
        return np.where(byte[..., None] == 255, np.nan, VALUES[code] * 2.0 ** (np.maximum(byte, 1)[..., None] - 127.0))


def token_logprobs(x, token, temperature, top_n):
    """One row x [V] in 64 bits: (logprob, entropy, rank, ids, their log probabilities)."""
    t = x / temperature
    with np.errstate(all="ignore"):
        top = t.max()
        lse = top + np.log(np.exp(t - top).sum())
        lp = t - lse
        p = np.exp(lp)
        entropy = -np.where(p > 0, p * lp, 0.0).sum() if np.isfinite(lse) else np.nan
        ids = np.arange(x.size)
        rank = 1 + int(((x > x[token]) | ((x == x[token]) & (ids < token))).sum())
        good = ids[x > -np.inf]
        order = good[np.lexsort((good, -x[good]))][:top_n]
        ids = np.full(top_n, -1)
        best = np.full(top_n, -np.inf)
        ids[:order.size], best[:order.size] = order, lp[order]
    return lp[token], entropy, rank, ids, best
