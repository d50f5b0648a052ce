"""Plain fp64 statements of the draft-tree operators (numpy, one entry at a time where that is clearest).

Test infrastructure: it shares no code with the CUDA path.  T nodes a tree; D = 128 channels; P = 16 tokens a block.
"""

import math

import numpy as np

P = 16


def tree_layout(parent, n_nodes, ctx_len):
    """(mask uint64 [B, T], pos int32 [B, T]); padding nodes get 0 and ctx_len."""
    B, T = parent.shape
    mask, pos = np.zeros((B, T), np.uint64), np.zeros((B, T), np.int32)
    for b in range(B):
        for j in range(T):
            pos[b, j] = ctx_len[b]
            if j >= n_nodes[b]:
                continue
            word, depth, k = 1 << j, 0, int(parent[b, j])
            while k >= 0:
                word, depth, k = word | 1 << k, depth + 1, int(parent[b, k])
            mask[b, j], pos[b, j] = word, ctx_len[b] + depth
    return mask, pos


def qk_norm_rope(rows, hq, hkv, wq, wk, eps, inv_freq, pos):
    """rows [B, T, (hq + 2 hkv), D] -> q [B, T, hq, D], k and v [B, hkv, T, D]."""
    def one(x, w):
        if w is not None:
            x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
        a = (pos.astype(np.float64)[..., None] * inv_freq.astype(np.float64))[:, :, None]
        lo, hi = x[..., :64], x[..., 64:]
        return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)

    q, k = one(rows[:, :, :hq], wq), one(rows[:, :, hq:hq + hkv], wk)
    return q, k.transpose(0, 2, 1, 3), rows[:, :, hq + hkv:].transpose(0, 2, 1, 3)


def tree_attention(q, pool_k, pool_v, slot_table, ctx_len, k_tree, v_tree, mask, scale):
    """out [B, T, Hq, D], lse [B, T, Hq]: row (j, h) over the valid tokens of the occupied slots and the nodes of mask[b, j]."""
    B, T, Hq, D = q.shape
    Hkv = slot_table.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    for b in range(B):
        for h in range(Hkv):
            keys, vals = [], []
            for s, blk in enumerate(slot_table[b, h]):
                nv = min(P, int(ctx_len[b]) - int(blk) * P) if blk >= 0 else 0
                if nv > 0:
                    keys.append(pool_k[b, h, s, :nv])
                    vals.append(pool_v[b, h, s, :nv])
            ck = np.concatenate(keys) if keys else np.zeros((0, D))
            cv = np.concatenate(vals) if vals else np.zeros((0, D))
            for j in range(T):
                seen = [i for i in range(T) if int(mask[b, j]) >> i & 1]
                if not seen:
                    continue
                kk, vv = np.concatenate([ck, k_tree[b, h, seen]]), np.concatenate([cv, v_tree[b, h, seen]])
                x = kk @ q[b, j, h * G:(h + 1) * G].T * scale                     # [tokens, G]
                m = x.max(0)
                with np.errstate(invalid="ignore"):                               # (an infinite score: NaN)
                    e = np.exp(x - m)
                out[b, j, h * G:(h + 1) * G] = (e / e.sum(0)).T @ vv
                lse[b, j, h * G:(h + 1) * G] = m + np.log(e.sum(0))
    return out, lse


def _clean(row):
    row = np.asarray(row, np.float64)
    return np.where(np.isfinite(row) & (row > 0), row, 0.0)


def verify_tree(probs, draft, tokens, parent, n_nodes, u_accept, u_sample):
    """(path [B, T], n_accept [B], next_token [B]); probs, draft: [B, T, V] (draft None: drafts not drawn at random)."""
    B, T, V = probs.shape
    path, count, token = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        if n_nodes[b] <= 0:
            continue
        cur, r, S = 0, _clean(probs[b, 0]), 1.0
        nodes = [0]
        for j in range(1, int(n_nodes[b])):
            x = int(tokens[b, j])
            if parent[b, j] != cur or not 0 <= x < V:
                continue
            d = _clean(draft[b, cur]) if draft is not None else None
            if r[x] > 0 and float(u_accept[b, j]) * S * (d[x] if d is not None else 1.0) < r[x]:
                cur, r, S = j, _clean(probs[b, j]), 1.0
                nodes.append(j)
            elif d is not None:
                r = np.maximum(r - S * d, 0.0)
                S = math.fsum(r)
            else:
                S -= r[x]
                r[x] = 0.0
        if not r.sum() > 0:
            r = _clean(probs[b, cur])
        path[b, :len(nodes)], count[b] = nodes, len(nodes)
        if r.sum() > 0:
            run = np.cumsum(r)
            over = np.nonzero((run > max(float(u_sample[b]), 0.0) * run[-1]) & (r > 0))[0]
            token[b] = over[0] if len(over) else np.nonzero(r)[0][-1]
    return path, count, token


def commit_path(host, pool, slot_table, kmin, kmax, k_tree, v_tree, path, n_accept, ctx_len):
    """Writes the accepted rows in place; returns ctx_len_out.  host [L, B, H, N, 2, P, D] (or None), pool [L, B, H, K, 2, P, D]
    (or None), slot_table [L, B, H, K], kmin / kmax [L, B, H, N, D], k_tree / v_tree [L, B, H, T, D]; any value type."""
    L, B, H, N = kmin.shape[:4]
    out = np.array(ctx_len, np.int32)
    for b in range(B):
        for i in range(int(n_accept[b])):
            n, t = divmod(int(ctx_len[b]) + i, P)
            if n >= N:
                break
            out[b] += 1
            node = int(path[b, i])
            for layer in range(L):
                for h in range(H):
                    k, v = k_tree[layer, b, h, node], v_tree[layer, b, h, node]
                    if host is not None:
                        host[layer, b, h, n, 0, t], host[layer, b, h, n, 1, t] = k, v
                    if pool is not None:
                        for s in np.nonzero(slot_table[layer, b, h] == n)[0]:
                            pool[layer, b, h, s, 0, t], pool[layer, b, h, s, 1, t] = k, v
                    kmin[layer, b, h, n] = k if t == 0 else np.minimum(kmin[layer, b, h, n], k)
                    kmax[layer, b, h, n] = k if t == 0 else np.maximum(kmax[layer, b, h, n], k)
    return out
