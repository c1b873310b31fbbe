"""Float64 oracle of the paged-cache serving operators: slots, append with head
norm and rotation, attention over pages, verification of drafted tokens.

Plain loops over sequences, tokens and pages, straight from the definitions;
numpy only."""

import numpy as np


def slots(cu_q, kv_len, table, page, total_q):
    """Position and slot of every packed row (0 and -1 for a row with no place)."""
    pos, slot = np.zeros(total_q, np.int64), np.full(total_q, -1, np.int64)
    for b in range(len(kv_len)):
        n = cu_q[b + 1] - cu_q[b]
        for i in range(n):
            p = kv_len[b] - n + i
            if p >= 0:
                pos[cu_q[b] + i] = p
                slot[cu_q[b] + i] = table[b][p // page] * page + p % page
    return pos, slot


def head_norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x, cos_sin, interleaved):
    """x [T, heads, d]; cos_sin [T, rot]: rot / 2 cosines, then the sines."""
    x = np.array(x, np.float64)
    rot = cos_sin.shape[-1]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = cos_sin[:, None, i], cos_sin[:, None, rot // 2 + i]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * c - xb * s
        x[..., b] = xb * c + xa * s
    return x


def gather(cache, table_row, page, kv):
    """The first kv rows of a sequence: [kv, Hkv, d] out of [pages, page, Hkv, d]."""
    return np.stack([cache[table_row[j // page], j % page] for j in range(kv)]) if kv else \
        np.zeros((0,) + cache.shape[2:])


def attention(q, keys, values, scale, causal):
    """One sequence: q [n, H, d], keys, values [kv, Hkv, d] -> o [n, H, d], lse
    [n, H], weight [n, H, d] = sum_j p_j |v_j|, reach [n, H] = the largest
    scale * sum |q| |k| over the visible keys (the scale of rounding errors)."""
    n, H, d = q.shape
    kv, Hkv, _ = keys.shape
    o, w = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, reach = np.full((n, H), -np.inf), np.zeros((n, H))
    for h in range(H):
        k, v = keys[:, h // (H // Hkv)], values[:, h // (H // Hkv)]
        for i in range(n):
            m = min(kv, kv - n + i + 1) if causal else kv
            if m <= 0:
                continue
            s = scale * (k[:m] @ q[i, h])
            top = s.max()
            e = np.exp(s - top)
            lse[i, h] = top + np.log(e.sum())
            p = e / e.sum()
            o[i, h] = p @ v[:m]
            w[i, h] = p @ np.abs(v[:m])
            reach[i, h] = scale * (np.abs(k[:m]) @ np.abs(q[i, h])).max()
    return o, lse, w, reach


def _softmax(x, temperature):
    z = np.asarray(x, np.float64) / temperature
    e = np.exp(z - z.max())
    return e / e.sum()


def verify(target, draft, tokens, u, expo, n, temperature):
    """One sequence: target [S + 1, V], draft [S, V] or None, tokens [S], u [S],
    expo [V], n drafts -> (out [S + 1], accepted, margin). margin is the least
    relative distance of any decision from its border, in units of the terms
    compared: relative errors in p and q below it cannot change the result."""
    S, V = len(tokens), target.shape[1]
    out, margin = np.full(S + 1, -1, np.int64), np.inf
    for at in range(n + 1):
        drafted = at < n
        if temperature == 0:
            choice = int(np.argmax(target[at]))
            if drafted and tokens[at] == choice:
                out[at] = tokens[at]
                continue
            out[at] = choice
            return out, at, margin
        p = _softmax(target[at], temperature)
        w, size = p, p
        if drafted:
            x = tokens[at]
            if draft is None:
                q = (np.arange(V) == x).astype(np.float64)
            else:
                q = _softmax(draft[at], temperature)
            left, right = u[at] * q[x], p[x]
            if left + right > 0:
                margin = min(margin, abs(left - right) / (left + right))
            if left < right:
                out[at] = x
                continue
            if (p > q).any():
                w, size = np.maximum(p - q, 0), np.where(p > q, p + q, 0)
                if draft is None:
                    size = w
        score, size = w / expo, size / expo
        choice = int(np.argmax(score))
        # smallest t with score_c - t size_c <= score_j + t size_j for some j
        gap = (score[choice] - score) / (size[choice] + size + 1e-300)
        gap[choice] = np.inf
        if V > 1:
            margin = min(margin, gap.min())
        out[at] = choice
        return out, at, margin
