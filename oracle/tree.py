"""Float64 oracle of the calls on trees of drafted tokens: masks and positions,
attention by mask, verification, commit.  Sequences, locations and cache as in
``mla.py``; parents are indices within a sequence, -1 for none."""

import numpy as np

from .mla import NEG_INF, context_row


def ancestors(parents):
    """Of each node of one sequence: the list of its ancestors and itself, from
    the root on (an invalid parent counts as none)."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def layout(parents, query_start_loc, seq_lens, words: int):
    """(mask [T, words] of Python integers as int64 values, positions [T])."""
    T = len(parents)
    mask, pos = np.zeros((T, words), dtype=np.int64), np.zeros(T, dtype=np.int64)
    for r, n in enumerate(seq_lens):
        lo, hi = int(query_start_loc[r]), int(query_start_loc[r + 1])
        for i, line in enumerate(ancestors(list(parents[lo:hi]))):
            for j in line:
                if j < 64 * words:
                    mask[lo + i, j // 64] |= np.array(1 << (j % 64), dtype=np.uint64).astype(np.int64)
            pos[lo + i] = int(n) - (hi - lo) + len(line) - 1
    return mask, pos


def bit(row, j: int) -> bool:
    """Bit j of one token's mask (int64 words)."""
    return j // 64 < len(row) and bool((int(row[j // 64]) >> (j % 64)) & 1)


def tree_attention(q_latent, cache, block_table, query_start_loc, seq_lens, mask, dims):
    """mla.latent_attention with masks: a token sees all positions before its
    sequence's new tokens, and new token j where bit j of its mask is set."""
    q = np.asarray(q_latent, dtype=np.float64)
    T, H, _ = q.shape
    L = dims.kv_lora_rank
    o, lse = np.full((T, H, L), np.nan), np.full((H, T), np.nan)
    mass, size = np.zeros((T, H, L)), np.zeros((H, T))
    for r, n in enumerate(seq_lens):
        lo, hi = int(query_start_loc[r]), int(query_start_loc[r + 1])
        base = int(n) - (hi - lo)
        for t in range(lo, hi):
            sees = [j for j in range(max(0, int(n))) if j < base or bit(mask[t], j - base)]
            if not sees:
                o[t], lse[:, t] = 0.0, NEG_INF
                continue
            c = np.stack([context_row(cache, block_table, r, j, dims.block_size)
                          for j in sees]).astype(np.float64)
            s = q[t] @ c.T * dims.softmax_scale
            size[:, t] = (np.abs(q[t]) @ np.abs(c).T).max(axis=1) * dims.softmax_scale
            mx = s.max(axis=1, keepdims=True)
            e = np.exp(s - mx)
            tot = e.sum(axis=1, keepdims=True)
            lse[:, t] = (mx + np.log(tot))[:, 0]
            o[t] = (e / tot) @ c[:, :L]
            mass[t] = (e / tot) @ np.abs(c[:, :L])
    return o, lse, mass, size


def verify(target, draft, tokens, parents, uniform, u_next, most: int, slack=None):
    """One sequence: (kept nodes, next token).  target, draft [n, V]; draft None:
    chosen children; uniform None: greedy.  With slack, a third value: the
    tokens with mass whose share of the sum comes within slack of the next
    token's border, slack being a part of the row before anything was taken out
    and divided by its sum."""
    n, V = target.shape
    if n == 0:
        return ([], -1) if slack is None else ([], -1, [-1])
    p64 = np.asarray(target, dtype=np.float64)
    up = [p if 0 <= p < i else -1 for i, p in enumerate(parents)]
    cur, path = 0, [0]
    while True:
        kids = [i for i in range(n) if up[i] == cur and i > cur and 0 <= tokens[i] < V]
        if len(path) >= most:
            kids = []
        if uniform is None:
            row = np.where(np.isnan(p64[cur]), -np.inf, p64[cur])
            best = int(row.argmax())
            kids = [i for i in kids if tokens[i] == best]
            if not kids:
                return (path, best) if slack is None else (path, best, [best])
            cur = kids[0]
            path.append(cur)
            continue
        p = np.maximum(np.nan_to_num(p64[cur], nan=0.0), 0.0)
        left, mass, kept, scale = p, 1.0, None, 1.0
        for i in kids:
            x = tokens[i]
            q = 1.0 if draft is None else float(draft[cur][x])
            if float(uniform[i]) * q * mass < left[x]:
                kept = i
                break
            if draft is None:
                left = left.copy()
                left[x] = 0.0
            elif mass > 0:
                scale *= mass
                left = np.maximum(left / mass - np.asarray(draft[cur], dtype=np.float64), 0.0)
            mass = left.sum()
        if kept is None:
            total = np.cumsum(left if left.sum() > 0 else p)
            border = float(u_next) * total[-1]
            v = min(int(np.searchsorted(total, border, side="right")), V - 1)
            if slack is None:
                return path, v
            e, own = slack / scale, np.diff(total, prepend=0.0)
            near = (own > 0) & (total > border - e) & (total - own <= border + e)
            return path, v, sorted({v, *(int(x) for x in np.flatnonzero(near))})
        cur = kept
        path.append(cur)


def commit(cache, block_table, query_start_loc, seq_lens, path, kept, block_size: int):
    """Moves the rows of one layer's cache in place; returns the new lengths."""
    lens = []
    for r, n in enumerate(seq_lens):
        m = int(query_start_loc[r + 1]) - int(query_start_loc[r])
        base = max(0, int(n)) - m

        def slot(j):
            return int(block_table[r][j // block_size]), j % block_size

        k = max(0, min(int(kept[r]), m, len(path[r])))
        moves = [(base + int(path[r][d]), base + d) for d in range(k)
                 if d < int(path[r][d]) < m and base + d >= 0]
        rows = [cache[slot(a)].copy() for a, _ in moves]
        for row, (_, b) in zip(rows, moves):
            cache[slot(b)] = row
        lens.append(max(0, base + k))
    return lens
