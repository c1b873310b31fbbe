"""Float64 oracle of the operators around trees of drafted tokens: masks and
positions of a tree's nodes, attention under a mask, sampling with limits, the
walk along drawn tokens, kept rows moved together, and pages shared, handed out
and taken back by their counts of owners.

Plain loops, straight from the definitions; numpy only."""

import numpy as np


def mask(parents):
    """[n, n] truth values: node i sees node j (itself and its ancestors)."""
    n = len(parents)
    m = np.zeros((n, n), bool)
    for i in range(n):
        p = i
        while p >= 0:
            m[i, p] = True
            p = parents[p]
    return m


def depths(parents):
    return mask(parents).sum(1) - 1


def words(m, count):
    """Truth values [n, nodes] as bits of int64 words [n, count]."""
    out = np.zeros((m.shape[0], count), np.uint64)
    for i, j in zip(*np.nonzero(m)):
        out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def attention(q, keys, values, scale, seen):
    """One sequence: q [n, H, d], keys, values [kv, Hkv, d], seen [n, kv] -> o [n, H,
    d], lse [n, H], weight [n, H, d] = sum_j p_j |v_j|, reach [n, H] = the largest
    scale * sum |q| |k| over the visible keys."""
    n, H, d = q.shape
    Hkv = keys.shape[1]
    o, w = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, reach = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        j = np.nonzero(seen[i])[0]
        if len(j) == 0:
            continue
        for h in range(H):
            k, v = keys[j, h // (H // Hkv)], values[j, h // (H // Hkv)]
            s = scale * (k @ q[i, h])
            top = s.max()
            e = np.exp(s - top)
            lse[i, h] = top + np.log(e.sum())
            p = e / e.sum()
            o[i, h], w[i, h] = p @ v, p @ np.abs(v)
            reach[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return o, lse, w, reach


def accept(parents, tokens, sampled):
    """The walk from node 0: (nodes, tokens drawn at them)."""
    path, at = [], 0
    while at is not None and at < len(parents):
        path.append(at)
        nxt = None
        for j in range(at + 1, len(parents)):
            if parents[j] == at and tokens[j] == sampled[at] and sampled[at] >= 0:
                nxt = j
                break
        at = nxt
    return path, [sampled[i] for i in path]


def kept(logits, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """What the limits leave of a row: (indices in descending order, their weights
    exp((x - max) / T), and the least relative distance of top_p's sums from its
    border and of the weights from min_p's: errors below it move no border)."""
    x = np.asarray(logits, np.float64)
    order = np.argsort(-x, kind="stable")
    order = order[np.isfinite(x[order])]
    w = np.exp((x[order] - x[order[0]]) / temperature)
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    margin = np.inf
    if top_p < 1:
        run = np.cumsum(w)
        n = max(1, int((run - w < max(top_p, 0.0) * run[-1]).sum()))
        if top_p > 0:
            margin = np.abs(run / run[-1] - top_p).min()
        order, w = order[:n], w[:n]
    if min_p > 0:
        keep = w >= min(min_p, 1.0)
        margin = min(margin, np.abs(w / min(min_p, 1.0) - 1)[1:].min(initial=np.inf))
        order, w = order[keep], w[keep]
    return order, w, margin


def sample(logits, expo, temperature, top_k=0, top_p=1.0, min_p=0.0, draw_alone=False):
    """One row: (token, log-probability, margin): margin is the least relative
    distance of the draw, or (unless draw_alone) of a limit, from its border."""
    x = np.asarray(logits, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
        return -1, np.nan, np.inf
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, np.inf
    idx, w, margin = kept(x, temperature, top_k, top_p, min_p)
    if draw_alone:
        margin = np.inf
    score = w / np.asarray(expo, np.float64)[idx]
    best = score.max()
    token = int(idx[score == best].min())
    rest = score[idx != token]
    if len(rest):
        margin = min(margin, 1 - rest.max() / best if rest.max() < best else np.inf)
    return token, float(np.log(w[list(idx).index(token)] / w.sum())), margin


def compact(cache, table, page, keep, base):
    """In place, one sequence: row base + keep[i] to row base + i."""
    rows = [cache[table[(base + k) // page], (base + k) % page].copy() for k in keep]
    for i, r in enumerate(rows):
        cache[table[(base + i) // page], (base + i) % page] = r


def pages(length, page):
    return -(-length // page)


def fork(table, lens, src, out, refs, page):
    """In place (out, refs); the new rows' lengths."""
    for i, s in enumerate(src):
        for j in range(pages(lens[s], page)):
            out[i][j] = table[s][j]
            refs[table[s][j]] += 1
    return [lens[s] for s in src]


def grow(table, lens, new, refs, page):
    """In place (table, refs) -> (copy_src, copy_dst, pages left; below 0: missing,
    and nothing changed)."""
    n = len(lens)
    last = [table[i][lens[i] // page] if new[i] > lens[i] and lens[i] % page else -1
            for i in range(n)]
    shared = [p if p >= 0 and refs[p] > 1 else -1 for p in last]
    copied = [p >= 0 and shared[:i].count(p) < refs[p] - 1 for i, p in enumerate(shared)]
    wants = []
    for i in range(n):
        first = pages(lens[i], page) - copied[i]
        wants += [(i, j) for j in range(first, pages(new[i], page))]
    free = [p for p in range(len(refs)) if refs[p] == 0]
    src, dst = [-1] * n, [-1] * n
    if len(free) < len(wants):
        return src, dst, len(free) - len(wants)
    for (i, j), p in zip(wants, free):
        if copied[i] and j == pages(lens[i], page) - 1:
            src[i], dst[i] = shared[i], p
            refs[shared[i]] -= 1
        table[i][j] = p
        refs[p] = 1
    return src, dst, len(free) - len(wants)


def release(table, lens, refs, page, new=None):
    """In place (refs)."""
    for i in range(len(lens)):
        for j in range(pages(new[i] if new is not None else 0, page), pages(lens[i], page)):
            refs[table[i][j]] -= 1
