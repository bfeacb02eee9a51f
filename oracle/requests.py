"""Oracle of the operators of a server of many requests: low-rank adapters
beside a projection, sampling, attention for trees of drafted tokens and the
commit of an accepted branch.

Written from the definitions in 64 bits with plain loops; no code is shared
with the GPU path.  Inputs are numpy arrays of the exact values the device
holds.
"""

import numpy as np


def lora(x, y, adapters, a, b, scales, widths):
    """-> (out, reach): y + s B A x of each token's adapter, and what rounding
    errors scale with: for the first sum (s |B| (|A| |x|)) and for the second
    (s |B| |A x|)."""
    rank = b.shape[2]
    out = np.array(y, np.float64)
    first, second = np.zeros_like(out), np.zeros_like(out)
    for t, i in enumerate(adapters):
        if not 0 <= i < a.shape[0]:
            continue
        s = 1.0 if scales is None else float(scales[i])
        n = 0
        for j, w in enumerate(widths):
            down, up = a[i, j * rank:(j + 1) * rank], b[i, n:n + w]
            h = down @ x[t]
            out[t, n:n + w] += s * (up @ h)
            first[t, n:n + w] = abs(s) * (np.abs(up) @ (np.abs(down) @ np.abs(x[t])))
            second[t, n:n + w] = abs(s) * (np.abs(up) @ np.abs(h))
            n += w
    return out, first, second


def sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None):
    """One row -> (scores of all entries, probabilities): 0 where not kept.
    Without an entry both are all 0."""
    l = np.array(logits, np.float64)
    l[np.isnan(l)] = -np.inf
    l = l + 0.0
    n = len(l)
    none = np.zeros(n), np.zeros(n)
    order = np.argsort(-l, kind="stable")
    order = order[~np.isneginf(l[order])]
    if len(order) == 0:
        return none
    t = 1.0 if temperature is None else float(temperature)
    if not t > 0:
        order, t = order[:1], 1.0
        top_k = top_p = min_p = None
    t = max(t, float(np.float32(1e-6)))
    top = l[order[0]]
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        w = np.exp((l[order] - top) / t) if np.isfinite(top) else (l[order] == top).astype(np.float64)
    if top_k is not None and int(top_k) > 0:
        order, w = order[:int(top_k)], w[:int(top_k)]
    if top_p is not None and float(top_p) < 1:
        before = np.cumsum(w) - w
        keep = max(1, int((before < max(float(top_p), 0.0) * w.sum()).sum()))
        order, w = order[:keep], w[:keep]
    if min_p is not None and float(min_p) > 0:
        keep = max(1, int((w >= min(float(min_p), 1.0)).sum()))
        order, w = order[:keep], w[:keep]
    scores, probs = np.zeros(n), np.zeros(n)
    scores[order] = w / np.asarray(noise, np.float64)[order]
    probs[order] = w / w.sum()
    return scores, probs


def tree_attention(q, k, v, page_table, seq_lens, cu_q, sees, page_size, scale, k_scale=None, v_scale=None):
    """-> dict as of oracle.serving.attention; sees: [tokens, words] bit masks
    over the new tokens of a sequence (uint64)."""
    T, H, D = q.shape
    kv_heads = k.shape[2]
    group = H // kv_heads
    out, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    weight, reach = np.zeros((T, H, D)), np.zeros((T, H))
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(cu_q[b + 1] - cu_q[b])
        rows = np.arange(L)
        pages = page_table[b][rows // page_size] if L else np.zeros(0, int)
        for t in range(n):
            tok = int(cu_q[b]) + t
            seen = []
            for j in range(L):
                node = j - (L - n)
                if node < 0 or (int(sees[tok][node // 64]) >> (node % 64)) & 1:
                    seen.append(j)
            for h in range(kv_heads):
                kk = np.asarray(k[pages[seen], rows[seen] % page_size, h], np.float64) * (1.0 if k_scale is None else float(k_scale[h]))
                vv = np.asarray(v[pages[seen], rows[seen] % page_size, h], np.float64) * (1.0 if v_scale is None else float(v_scale[h]))
                for head in range(h * group, (h + 1) * group):
                    if not seen:
                        out[tok, head], lse[tok, head] = 0.0, -np.inf
                        continue
                    x = np.asarray(q[tok, head], np.float64)
                    s = scale * (kk @ x)
                    m = s.max()
                    e = np.exp(s - m)
                    out[tok, head] = (e @ vv) / e.sum()
                    lse[tok, head] = m + np.log(e.sum())
                    weight[tok, head] = (e @ np.abs(vv)) / e.sum()
                    reach[tok, head] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
    return dict(out=out, lse=lse, weight=weight, reach=reach)


def tree_commit(tokens, parents, sampled, cu, seq_lens, depth):
    """-> (out_tokens [batch, depth + 1], accepted, new lengths, moves): moves of
    each sequence as (from, to) positions."""
    out, accepted, lens, moves = [], [], [], []
    for b in range(len(seq_lens)):
        first, n, L = int(cu[b]), int(cu[b + 1] - cu[b]), int(seq_lens[b])
        row, node, path = [], 0, []
        while n:
            draw = int(sampled[first + node])
            row.append(draw)
            below = [i for i in range(node + 1, n) if parents[first + i] == node and tokens[first + i] == draw]
            if len(path) == depth or not below:
                break
            node = below[0]
            path.append(node)
        out.append(row + [-1] * (depth + 1 - len(row)))
        accepted.append(len(path))
        lens.append(L - n + 1 + len(path) if n else L)
        moves.append([(L - n + i, L - n + d) for d, i in enumerate(path, 1)])
    return np.array(out, np.int32), np.array(accepted, np.int32), np.array(lens, np.int32), moves
