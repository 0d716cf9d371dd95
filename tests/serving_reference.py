"""Plain 64-bit forms of the target-side operators (numpy, CPU), written from their formulas, and
the error bounds that the tests hold the kernels to.

Bounds.  A value rounded to bf16 (8 significant bits) is off by at most 2^-8 of itself.  An
attention output rounds each weight p_j to bf16 and then the sum: with A = sum_j p_j |v_j| the
error is at most (2^-8 + 2^-8) A, and the fp32 scores (D products of unit-size numbers, error of the
score well below 5e-5) add a relative 1e-4 at most."""
import numpy as np

BF16 = 2.0 ** -8


def rotate(x, cos, sin, interleaved):
    """x [.., D] by the angles of cos, sin [.., rot / 2]."""
    x = np.array(x, np.float64)
    half = cos.shape[-1]
    a_at, b_at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., a_at].copy(), x[..., b_at].copy()
    x[..., a_at], x[..., b_at] = a * cos - b * sin, b * cos + a * sin
    return x


def attention(q, keys, vals, ctx, scale, window, n_sink):
    """One request: q [n, Hq, D], keys / vals [ctx + n, Hkv, D].  Returns out, lse and A (see above)."""
    n, hq, d = q.shape
    g = hq // keys.shape[1]
    out, lse, mag = np.zeros((n, hq, d)), np.zeros((n, hq)), np.zeros((n, hq, d))
    for i in range(n):
        p = ctx + i
        j = np.arange(p + 1)
        if window:
            j = j[(j > p - window) | (j < n_sink)]
        for h in range(hq):
            s = scale * (keys[j, h // g] @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            lse[i, h] = m + np.log(w.sum())
            w /= w.sum()
            out[i, h] = w @ vals[j, h // g]
            mag[i, h] = w @ np.abs(vals[j, h // g])
    return out, lse, mag


def attention_bound(mag):
    return mag * (2 * BF16 + 1e-4) + 1e-30


def logit_rules(logits, ids, count, prompt, rho, freq, pres, bias, mask):
    """One request: logits [n, V], ids [n], count / prompt [V], bias [V], mask [n, V] bool.  Returns the
    rows and the size of the terms that fp32 rounds."""
    out, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    count = count.astype(np.int64).copy()
    for i in range(logits.shape[0]):
        if i and 0 <= ids[i] < count.size:
            count[ids[i]] += 1
        l = logits[i].astype(np.float64)
        seen = prompt | (count > 0)
        with np.errstate(invalid="ignore"):
            l = np.where(seen, np.where(l > 0, l / rho, l * rho), l)
            mag[i] = np.abs(l) + np.abs(freq * count) + np.abs(pres) + np.abs(bias)
            l = l - freq * count - pres * (count > 0) + bias
        out[i] = np.where(mask[i], l, -np.inf)
    return out, mag


def history_words(prompt_ids, said_ids, V):
    count = np.bincount(np.asarray(said_ids, np.int64), minlength=V)[:V] if len(said_ids) else np.zeros(V, np.int64)
    flag = np.zeros(V, np.int64)
    flag[np.asarray(prompt_ids, np.int64)] = 1
    return (np.minimum(count, 32767) - 32768 * flag).astype(np.int16)
