"""Oracle of the serving operators: per-head norm and rotation, append to a
paged cache, attention over it, draft verification.

Written from the definitions in 64 bits with plain loops over tokens, heads and
sequences; no code is shared with the GPU path.  Inputs are numpy arrays of the
exact values the device holds (bf16 and E4M3 values as float64).
"""

import numpy as np


def norm_rope(x, weight, positions, table, rot, interleaved, eps):
    """[tokens, heads, dim] values -> (y, size): the normalised and rotated
    heads, and |n_a| + |n_b| of each output's pair (what rounding errors scale
    with)."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    y, size = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        known = 0 <= positions[t] < (table.shape[0] if table is not None else 1 << 62)
        for h in range(H):
            n = x[t, h]
            if weight is not None:
                n = n * np.asarray(weight, np.float64) / np.sqrt(np.mean(n * n) + eps)
            out, s = n.copy(), np.abs(n)
            if rot:
                half = rot // 2
                if not known:
                    out[:] = np.nan
                else:
                    cos = np.asarray(table[positions[t], :half], np.float64)
                    sin = np.asarray(table[positions[t], half:rot], np.float64)
                    a = np.arange(half) * 2 if interleaved else np.arange(half)
                    b = a + 1 if interleaved else a + half
                    out[a] = n[a] * cos - n[b] * sin
                    out[b] = n[b] * cos + n[a] * sin
                    s[a] = s[b] = np.abs(n[a]) + np.abs(n[b])
            y[t, h], size[t, h] = out, s
    return y, size


def attention(q, k, v, page_table, seq_lens, cu_q, page_size, scale, causal=True, window=0, k_scale=None, v_scale=None):
    """-> dict of out [tokens, heads, dim], lse, weight (sum_j p_j |v_j|) and
    reach (max_j scale sum_d |q_d k_jd|) of every row; rows outside cu_q are NaN.
    k, v: [pages, page_size, kv_heads, dim] values of the codes."""
    T, H, D = q.shape
    kv_heads = k.shape[2]
    group = H // kv_heads
    out = np.full((T, H, D), np.nan)
    lse = np.full((T, H), np.nan)
    weight, reach = np.zeros((T, H, D)), np.zeros((T, H))
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(cu_q[b + 1] - cu_q[b])
        rows = np.arange(L)
        pages = page_table[b][rows // page_size] if L else np.zeros(0, int)
        for h in range(kv_heads):
            kk = np.asarray(k[pages, rows % page_size, h], np.float64) * (1.0 if k_scale is None else float(k_scale[h]))
            vv = np.asarray(v[pages, rows % page_size, h], np.float64) * (1.0 if v_scale is None else float(v_scale[h]))
            for t in range(n):
                p = L - n + t
                hi = min(L, max(0, p + 1)) if causal else L
                lo = max(0, p - window + 1) if window else 0
                for g in range(group):
                    tok, head = int(cu_q[b]) + t, h * group + g
                    if lo >= hi:
                        out[tok, head], lse[tok, head] = 0.0, -np.inf
                        continue
                    x = np.asarray(q[tok, head], np.float64)
                    s = scale * (kk[lo:hi] @ x)
                    m = s.max()
                    e = np.exp(s - m)
                    out[tok, head] = (e @ vv[lo:hi]) / e.sum()
                    lse[tok, head] = m + np.log(e.sum())
                    weight[tok, head] = (e @ np.abs(vv[lo:hi])) / e.sum()
                    reach[tok, head] = (np.abs(kk[lo:hi]) @ np.abs(x)).max() * abs(scale)
    return dict(out=out, lse=lse, weight=weight, reach=reach)


def verify(target, draft, tokens, cu, uniforms, noise, max_drafts):
    """-> (out_tokens [batch, max_drafts + 1], accepted [batch]).  The
    comparisons are those of the binary32 definition: one rounded product,
    difference and quotient each.  A NaN probability counts as 0."""
    f32 = np.float32
    target = np.where(np.isnan(target), f32(0), target)
    draft = None if draft is None else np.where(np.isnan(draft), f32(0), draft)
    batch, vocab = noise.shape
    out, accepted = np.full((batch, max_drafts + 1), -1, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        first, n = int(cu[b]), int(cu[b + 1] - cu[b])
        k = 0
        while k < n:
            x = int(tokens[first + k])
            if not 0 <= x < vocab:
                break
            qx = f32(1) if draft is None else f32(draft[first + k, x])
            if not f32(uniforms[first + k]) * qx < f32(target[first + k + b, x]):
                break
            k += 1
        p = target[first + k + b].astype(f32)
        w = p
        if k < n:
            q = np.zeros(vocab, f32)
            if draft is not None:
                q = draft[first + k].astype(f32)
            elif 0 <= tokens[first + k] < vocab:
                q[tokens[first + k]] = 1
            w = np.where(p - q > 0, p - q, f32(0))
            if not (w > 0).any():
                w = p
        with np.errstate(divide="ignore", invalid="ignore"):
            score = w.astype(f32) / noise[b].astype(f32)
        score = np.where(score > 0, score, f32(0))
        out[b, :k] = tokens[first:first + k]
        out[b, k] = int(np.argmax(score))
        accepted[b] = k
    return out, accepted
