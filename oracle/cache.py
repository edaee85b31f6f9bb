"""Rotary positions, the 8-bit cache and attention over it (oracle, fp64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Plain loops over the
definitions; pages are looked up token by token.
"""

import numpy as np

from .rpbh import hadamard, rotate

E_MIN, E_MAX = -40, 40


def rope(x, pos, freq, axis, halves, inverse=False):
    """x [T, heads, d] float64, pos int [T, axes] -> turned rows."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    n = len(freq)
    for p in range(n):
        i, j = (p, p + n) if halves else (2 * p, 2 * p + 1)
        phi = pos[:, axis[p]].astype(np.float64) * freq[p]
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None] * (-1 if inverse else 1)
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    return y


def turn(x, rot):
    """Pi x for rows x; rot = (perm, signs, block) or None."""
    return np.asarray(x, dtype=np.float64) if rot is None else rotate(x, *rot)


def turn_back(u, rot):
    """Pi^T u."""
    if rot is None:
        return np.asarray(u, dtype=np.float64)
    perm, signs, h = rot
    H = hadamard(h)
    z = np.concatenate([u[..., i:i + h] @ H for i in range(0, u.shape[-1], h)], -1) * signs
    x = np.empty_like(z)
    x[..., perm] = z
    return x


def step_exponent(amax):
    """Least e in [E_MIN, E_MAX] with amax <= 127 * 2^e (E_MAX if there is none)."""
    for e in range(E_MIN, E_MAX):
        if amax <= 127 * 2.0 ** e:
            return e
    return E_MAX


def write(codes, exps, rows, cu, past, table, rot):
    """Writes rows [T, heads, d] into codes int [pages, heads, page, d] and exps
    int [pages, heads], in place.  Returns the distance of each written value
    from the nearest border between two codes, [T, heads, d] (in steps)."""
    P = codes.shape[2]
    u = turn(rows, rot)
    near = np.full(u.shape, np.inf)
    for b in range(len(past)):
        n = cu[b + 1] - cu[b]
        places = [(past[b] + i) for i in range(n)]
        for slot in sorted({p // P for p in places}):
            page, held = table[b][slot], max(0, min(past[b] - slot * P, P))
            mine = [i for i, p in enumerate(places) if p // P == slot]
            for h in range(codes.shape[1]):
                rows_h = u[[cu[b] + i for i in mine], h]
                e = step_exponent(np.abs(rows_h).max())
                if held:
                    was = exps[page, h]
                    e = max(e, was)
                    codes[page, h, :held] = np.rint(codes[page, h, :held] / 2.0 ** (e - was))
                exps[page, h] = e
                for i, r in zip(mine, rows_h):
                    t = r / 2.0 ** e
                    codes[page, h, places[i] % P] = np.clip(np.rint(t), -127, 127)
                    near[cu[b] + i, h] = np.abs(t - np.floor(t) - 0.5)
    return near


def gather(codes, scale, seq_table, n):
    """Values (rotated coordinates) of the first n tokens: [n, heads, d]."""
    P = codes.shape[2]
    out = np.zeros((n, codes.shape[1], codes.shape[3]))
    for t in range(n):
        page = seq_table[t // P]
        out[t] = codes[page, :, t % P].astype(np.float64) * scale[page].astype(np.float64)[:, None]
    return out


def lost_weights(p, vv, shift, step=None):
    """Bound, for each coordinate, of what the sum of p_j v_j loses below fp16's
    normal numbers.  A weight p_j 2^ev_j beside the row's largest, which stands at
    2^shift or above, is off by 2^-25 at most, and never by more than itself:
    min(p_j |v_j|, 2^-(25 + shift) M |v_j| / 2^ev_j) with M the largest p_j 2^ev_j.
    step: 2^ev_j; without it the values tell that codes are whole and at most 127:
    |v_j| / 2^ev_j <= 127 |v_j| / max |v_j|, 2^ev_j <= the least |v_j| but 0 (a key
    of nothing else: the largest of the others')."""
    a = np.abs(vv)
    if step is None:
        code = 127 * a / np.maximum(a.max(1, keepdims=True), 1e-300)
        step = np.where(a > 0, a, np.inf).min(1)
        if not np.isfinite(step).any():
            return np.zeros(vv.shape[1])
        step = np.where(np.isfinite(step), step, step[np.isfinite(step)].max())
    else:
        code = a / step[:, None]
    return np.minimum(p[:, None] * a, 2.0 ** -(25 + shift) * (p * step).max() * code).sum(0)


def attention(q, k, v, causal, scale, rot, empty=None, shift=0, step=None):
    """One sequence: q [n, heads, d]; k, v [len, kv heads, d] in rotated
    coordinates; empty [len, kv heads]: keys that count as absent.  Returns the
    output, and for every row a bound of its error's 2-norm from queries and
    weights that are rounded to half a step of fp16 (2^-12 of each):
    a score is off by ds <= 2^-12 scale sum |q||k|, a weight by a factor
    exp(+-2 max ds) (its own score and the sum) and by 2^-12, and by what weights
    below fp16's normal numbers lose (lost_weights; shift: where a row's largest
    weight stands at least, 2^shift; step [len, kv heads]: the values' scales)."""
    n, H, d = q.shape
    L, Hk, _ = k.shape
    u = turn(q, rot)
    out, bound = np.zeros(q.shape), np.zeros((n, H))
    for i in range(n):
        seen = max(0, L - n + i + 1) if causal else L
        for h in range(H):
            kh = h * Hk // H
            ok = np.ones(seen, bool) if empty is None else ~empty[:seen, kh]
            kk, vv = k[:seen, kh][ok], v[:seen, kh][ok]
            if not len(kk):
                continue
            s = scale * kk @ u[i, h]
            p = np.exp(s - s.max())
            p /= p.sum()
            # values of a query below 2^-14 of its largest are rounded to multiples of 2^-24
            ds = abs(scale) * (np.abs(kk) @ (2.0 ** -12 * np.abs(u[i, h]) + 2.0 ** -25 * np.abs(u[i, h]).max()))
            rel = np.expm1(2 * ds[p > 1e-9].max()) + 2.0 ** -12 + 2.0 ** -18
            out[i, h] = turn_back((p @ vv)[None], rot)[0]
            bound[i, h] = rel * np.linalg.norm(p @ np.abs(vv)) + np.linalg.norm(
                lost_weights(p, vv, shift, None if step is None else step[:seen, kh][ok]))
    return out, bound
