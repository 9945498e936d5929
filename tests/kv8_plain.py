"""Plain 64-bit numpy forms of the attention operators, sequence by sequence and page by page."""
import numpy as np


def rope(x, weight, offset, eps, normalize, freq, pos, interleaved, scale):
    """x [T, H, D] float64; freq [R/2] radians a position.  Also the size that errors scale with."""
    y = x.astype(np.float64)
    if normalize:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        y = y * ((weight + offset) if weight is not None else 1.0)
    half = len(freq)
    ang = pos.astype(np.float64)[:, None] * freq
    c, s = np.cos(ang)[:, None] * scale, np.sin(ang)[:, None] * scale
    out, size = y.copy(), np.abs(y)
    a_at, b_at = ((np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved
                  else (np.arange(half), np.arange(half) + half))
    a, b = y[..., a_at], y[..., b_at]
    out[..., a_at], out[..., b_at] = a * c - b * s, a * s + b * c
    size[..., a_at] = size[..., b_at] = (np.abs(a) + np.abs(b)) * scale
    return out, size


def append(codes, amax, table, q_start, kv_len, x):
    """codes int8 [P, H, page, D], amax float64 [P, H], x float64 [T, H, D]; in place."""
    page = codes.shape[2]
    for b in range(len(kv_len)):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        p0, t = int(kv_len[b]) - (r1 - r0), r0
        while t < r1:
            pos = p0 + t - r0
            at, rows = pos % page, min(page - pos % page, r1 - t)
            pg = int(table[b, pos // page])
            for h in range(codes.shape[1]):
                new = x[t:t + rows, h]
                was = amax[pg, h] if at else 0.0
                now = max(was, np.abs(new).max())
                if now > was and at:
                    codes[pg, h, :at] = np.rint(codes[pg, h, :at].astype(np.float64) * was / now)
                codes[pg, h, at:at + rows] = np.rint(127.0 * new / now) if now > 0 else 0
                amax[pg, h] = now
            t += rows


def values(codes, amax, table_row, length):
    """[H, length, D] float64 of one sequence, its pages in order."""
    page = codes.shape[2]
    ids = table_row[:-(-length // page)]
    v = codes[ids].astype(np.float64) * amax[ids][:, :, None, None] / 127.0
    return v.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def attention(q, k, v, k_size, scale, causal, window):
    """One sequence: q [n, Hq, D], k, v [Hk, length, D].  Returns out, lse, and for the tolerance
    sum p |v| and max p a (a: the magnitude of the value's page, k_size [Hk, length]) and
    the largest sum |q k|."""
    n, hq, d = q.shape
    hk, length = k.shape[:2]
    g = hq // hk
    pos = length - n + np.arange(n)[:, None]
    j = np.arange(length)[None]
    see = (j <= pos) if causal else np.ones((n, length), bool)
    if window:
        see = see & (j > pos - window)
    out, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, top, reach = np.full((n, hq), -np.inf), np.zeros((n, hq)), np.zeros((n, hq))
    rows = see.any(1)
    for h in range(hq):
        if not rows.any():
            continue
        s = np.where(see, (q[:, h] @ k[h // g].T) * scale, -np.inf)[rows]
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        den = p.sum(1, keepdims=True)
        lse[rows, h] = (m + np.log(den))[:, 0]
        p /= den
        out[rows, h] = p @ v[h // g]
        size[rows, h] = p @ np.abs(v[h // g])
        top[rows, h] = (p * k_size[h // g]).max(1)
        reach[rows, h] = np.where(see[rows], (np.abs(q[rows, h]) @ np.abs(k[h // g]).T) * abs(scale), 0).max(1)
    return out, lse, size, top, reach
