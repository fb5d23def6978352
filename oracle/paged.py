"""Float64 (and whole-number) statement of the paged-cache operators."""

import numpy as np


def paged_block_tables(context, new, table, free, n_tokens, page):
    """Token by token: (slots, positions, cu_new, taken, table); -1 marks padding, and pages
    and slots that the free list has no page for."""
    table = np.array(table)
    slots, positions, cu, taken = [], [], [0], 0
    for r, (c, n) in enumerate(zip(context, new)):
        for p in range(c, c + n):
            if p % page == 0:
                table[r, p // page] = free[taken] if taken < len(free) else -1
                taken += 1
            i = table[r, p // page]
            slots.append(i * page + p % page if i >= 0 else -1)
            positions.append(p)
        cu.append(cu[-1] + n)
    pad = [-1] * (n_tokens - len(slots))
    return (np.array(slots + pad), np.array(positions + pad), np.array(cu), taken, table)


def paged_chunk_attention(q, k_cache, v_cache, table, cu, context, causal, page_mask=None,
                          scale=None):
    """q (Hq,T,D), caches (n_pages,Hkv,page,D), page_mask (R,Hkv,width) or None. Returns
    (out, spread): spread = sum_j weight_j |v_j|, the size that rounding the weights acts on."""
    Hq, T, D = q.shape
    _, Hkv, page, _ = k_cache.shape
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, spread = np.zeros((Hq, T, D)), np.zeros((Hq, T, D))
    for r in range(len(context)):
        t0, t1 = cu[r], cu[r + 1]
        length = context[r] + t1 - t0
        for g in range(Hkv):
            keys = [j for j in range(length)
                    if page_mask is None or page_mask[r, g, j // page]]
            if not keys:
                continue
            keys = np.array(keys)
            k = k_cache[table[r][keys // page], g, keys % page]
            v = v_cache[table[r][keys // page], g, keys % page]
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                for t in range(t0, t1):
                    see = keys <= context[r] + t - t0 if causal else np.ones(len(keys), bool)
                    if not see.any():
                        continue
                    s = scale * (k[see] @ q[h, t])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[h, t] = w @ v[see]
                    spread[h, t] = w @ np.abs(v[see])
    return out, spread
